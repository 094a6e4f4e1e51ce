// Residual step of a transformer block with the norms on either side of it, in one pass, and its
// gradient.
//
//   u = y * rsqrt(mean(y^2) + eps) * w_post     (or u = y without w_post)
//   h = x + scale * g * u                       (g: per channel, per token, or 1)
//   z = h * rsqrt(mean(h^2) + eps) * w_pre      (only with w_pre)
//
// Gradient, with r1, r2 the two reciprocal RMS values, yh = y r1, hh = h r2 and sums over a row:
//   dH = dh + r2 (dz w_pre - hh mean(dz w_pre hh))        dx = dH
//   du = scale g dH,  dg = scale u dH
//   dy = r1 (du w_post - yh mean(du w_post yh))           (or dy = du)
//   dw_pre = sum_t dz hh,  dw_post = sum_t du yh,  dg (per channel) = sum_t scale u dH
//
// Everything is HBM bound: a row is read once, the reductions run on it in fp32 and it is written
// once. Forward, a row belongs to a group of `wpr` warps, each lane holding VPT pieces of 8 columns in
// registers; a group of one warp needs shuffles only, larger ones (a whole block) meet in shared memory.
// 37007 x 1280 in bf16 takes 63 us (6.0 TB/s), what a plain copy of as many bytes takes (rows through a ring in
// shared memory, as the gradient has them, took 107 us). h is normalised before it is rounded to its storage type;
// the gradient recomputes r2 from the stored h it is given.
//
// The sums over tokens are accumulated in registers by persistent groups (a lane keeps its columns
// from row to row), written once per group as a partial row of the workspace and added up by a
// second small kernel in a fixed order, so results do not change from run to run.
#include <type_traits>

#include "internal.h"
#include "rope_math.cuh"
#include "sm100.cuh"

namespace vit {
namespace {

constexpr int kMaxWarps = 16;             // per row: up to 8192 columns, two pieces of 8 per lane

using rope::unpack8;

__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(rope::pack2(x[0], x[1]), rope::pack2(x[2], x[3]), rope::pack2(x[4], x[5]),
                      rope::pack2(x[6], x[7]));
}

// 8 consecutive values of a residual stream in bf16 or fp32
template <bool F32> struct Vec8;
template <> struct Vec8<false> {
    uint4 a;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        a = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
    }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float *x) const { unpack8(a, x); }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float *x) {
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) = pack8(x);
    }
};
template <> struct Vec8<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        a = s[0];
        b = s[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float *x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float *x) {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of v over a row's group: shuffles, then (for groups of several warps, each a whole block) the
// warps' sums through shared memory, added in warp order by every thread. `buf` alternates between
// two halves of `red` so that one barrier per reduction is enough.
__device__ __forceinline__ float row_sum(float v, int wpr, float *red, int &buf) {
    v = warp_sum(v);
    if (wpr == 1) return v;
    float *r = red + buf * kMaxWarps;
    buf ^= 1;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < wpr; ++w) s += r[w];
    return s;
}

struct Fwd {
    const void *x;
    const __nv_bfloat16 *y, *gate, *w_post, *w_pre;
    void *h;
    __nv_bfloat16 *z;
    int64_t T, x_stride, y_stride, gate_stride, h_stride, z_stride;
    int C;
    float scale, eps;
};

// ONE: a warp per row, whose lanes' places are constants (37007 x 1280: 63 us, 71 with the row's warps taken from
// the launch).
template <int VPT, bool F32, bool ONE>
__global__ void __launch_bounds__(ONE ? 128 : 512)
norm_residual_kernel(const Fwd p, int warps, int rows_per_block)
{
    const int wpr = ONE ? 1 : warps;
    __shared__ float s_red[2 * kMaxWarps];
    grid_wait();
    grid_release();
    const int lane_in_row = wpr == 1 ? (threadIdx.x & 31) : (int)threadIdx.x;
    const int row_in_block = wpr == 1 ? (int)(threadIdx.x >> 5) : 0;
    const int nvec = p.C >> 3, group = wpr * 32;
    const float inv_c = 1.f / (float)p.C;
    int buf = 0;
    for (int64_t t = (int64_t)blockIdx.x * rows_per_block + row_in_block; t < p.T;
         t += (int64_t)gridDim.x * rows_per_block) {
        Vec8<F32> vx[VPT];
        uint4 vy[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * group + lane_in_row;
            if (v < nvec) {
                vy[i] = *reinterpret_cast<const uint4 *>(p.y + t * p.y_stride + 8 * v);
                vx[i].load(p.x, t * p.x_stride + 8 * v);
            } else {
                vy[i] = make_uint4(0u, 0u, 0u, 0u);
                vx[i].zero();
            }
        }
        float r1 = 1.f;
        if (p.w_post) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float u[8];
                unpack8(vy[i], u);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
            }
            r1 = rsqrtf(row_sum(ss, wpr, s_red, buf) * inv_c + p.eps);
        }
        float h[VPT][8];
        float ss2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * group + lane_in_row;
            float u[8], x[8];
            unpack8(vy[i], u);
            vx[i].get(x);
            if (v < nvec) {
                if (p.w_post) {
                    float w[8];
                    unpack8(*reinterpret_cast<const uint4 *>(p.w_post + 8 * v), w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] *= r1 * w[e];
                }
                if (p.gate) {
                    float g[8];
                    unpack8(*reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride + 8 * v), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] *= g[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = fmaf(p.scale, u[e], x[e]);
                ss2 = fmaf(h[i][e], h[i][e], ss2);
            }
            if (v < nvec) Vec8<F32>::store(p.h, t * p.h_stride + 8 * v, h[i]);
        }
        if (!p.w_pre) continue;
        const float r2 = rsqrtf(row_sum(ss2, wpr, s_red, buf) * inv_c + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * group + lane_in_row;
            if (v >= nvec) continue;
            float w[8];
            unpack8(*reinterpret_cast<const uint4 *>(p.w_pre + 8 * v), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] *= h[i][e] * r2;
            *reinterpret_cast<uint4 *>(p.z + t * p.z_stride + 8 * v) = pack8(w);
        }
    }
}

struct Bwd {
    const __nv_bfloat16 *dz;
    const void *dh, *h;
    const __nv_bfloat16 *y, *gate, *w_post, *w_pre;
    void *dx;
    __nv_bfloat16 *dy, *dgate;     // dgate: per-token gate only
    float *part;                   // [groups][sums][C], in the order dw_pre, dw_post, dgate of those asked for
    int64_t T, dz_stride, dh_stride, h_stride, y_stride, gate_stride, dx_stride, dy_stride, dgate_stride;
    int C;
    int n_sum, at_pre, at_post, at_gate;   // how many sums, and each one's place (-1: not asked for)
    float scale, eps;
};

// Rows of at most 512 columns: one warp per row, straight from HBM into registers.
template <int VPT, bool F32>
__global__ void __launch_bounds__(256)
norm_residual_bwd_kernel(const Bwd p, int rows_per_block)
{
    grid_wait();
    grid_release();
    __shared__ float3 s_sum[256 * VPT];
    const int lane_in_row = threadIdx.x & 31, row_in_block = (int)(threadIdx.x >> 5);
    const int nvec = p.C >> 3, group = 32;
    const float inv_c = 1.f / (float)p.C;
    const bool gate_tok = p.gate && p.gate_stride != 0;
    float a_pre[VPT][8], a_post[VPT][8], a_gate[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) a_pre[i][e] = a_post[i][e] = a_gate[i][e] = 0.f;

    for (int64_t t = (int64_t)blockIdx.x * rows_per_block + row_in_block; t < p.T;
         t += (int64_t)gridDim.x * rows_per_block) {
        Vec8<F32> vdh[VPT], vh[VPT];
        uint4 vdz[VPT], vy[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * group + lane_in_row;
            vdh[i].zero();
            vh[i].zero();
            vdz[i] = vy[i] = make_uint4(0u, 0u, 0u, 0u);
            if (v < nvec) {
                if (p.w_pre) {
                    vh[i].load(p.h, t * p.h_stride + 8 * v);
                    vdz[i] = *reinterpret_cast<const uint4 *>(p.dz + t * p.dz_stride + 8 * v);
                }
                if (p.dh) vdh[i].load(p.dh, t * p.dh_stride + 8 * v);
                if (p.y) vy[i] = *reinterpret_cast<const uint4 *>(p.y + t * p.y_stride + 8 * v);
            }
        }
        // first reduction: sum h^2 and sum dz w_pre h
        float r2 = 0.f, c2 = 0.f;
        if (p.w_pre) {
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = i * group + lane_in_row;
                float h[8], dz[8], w[8];
                vh[i].get(h);
                unpack8(vdz[i], dz);
                unpack8(v < nvec ? *reinterpret_cast<const uint4 *>(p.w_pre + 8 * v) : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(h[e], h[e], ss);
                    dot = fmaf(dz[e] * w[e], h[e], dot);
                }
            }
            const float2 s = make_float2(warp_sum(ss), warp_sum(dot));
            r2 = rsqrtf(s.x * inv_c + p.eps);
            c2 = r2 * r2 * (s.y * inv_c);             // dH = dh + r2 (dz w - h c2)
        }
        float dH[VPT][8];
        float ssy = 0.f, doty = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * group + lane_in_row;
            vdh[i].get(dH[i]);
            if (v >= nvec) continue;
            if (p.w_pre) {
                float h[8], dz[8], w[8];
                vh[i].get(h);
                unpack8(vdz[i], dz);
                unpack8(*reinterpret_cast<const uint4 *>(p.w_pre + 8 * v), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dH[i][e] = fmaf(r2, fmaf(dz[e], w[e], -h[e] * c2), dH[i][e]);
                    a_pre[i][e] = fmaf(dz[e], h[e] * r2, a_pre[i][e]);
                }
            }
            Vec8<F32>::store(p.dx, t * p.dx_stride + 8 * v, dH[i]);
            if (p.w_post) {
                // second reduction: sum y^2 and sum du w_post y
                float y[8], w[8], g[8];
                unpack8(vy[i], y);
                unpack8(*reinterpret_cast<const uint4 *>(p.w_post + 8 * v), w);
                if (p.gate) unpack8(*reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride + 8 * v), g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float du = p.scale * dH[i][e] * (p.gate ? g[e] : 1.f);
                    ssy = fmaf(y[e], y[e], ssy);
                    doty = fmaf(du * w[e], y[e], doty);
                }
            }
        }
        float r1 = 1.f, c1 = 0.f;
        if (p.w_post) {
            const float2 s = make_float2(warp_sum(ssy), warp_sum(doty));
            r1 = rsqrtf(s.x * inv_c + p.eps);
            c1 = r1 * r1 * (s.y * inv_c);             // dy = r1 (du w - y c1)
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * group + lane_in_row;
            if (v >= nvec) continue;
            float y[8], w[8], g[8], dy[8], dg[8];
            unpack8(vy[i], y);
            if (p.gate) unpack8(*reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride + 8 * v), g);
            if (p.w_post) unpack8(*reinterpret_cast<const uint4 *>(p.w_post + 8 * v), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = p.scale * dH[i][e];
                const float du = p.gate ? d * g[e] : d;
                const float yh = y[e] * r1;
                dg[e] = d * (p.w_post ? yh * w[e] : y[e]);
                dy[e] = p.w_post ? r1 * fmaf(du, w[e], -y[e] * c1) : du;
                a_gate[i][e] += dg[e];
                a_post[i][e] = fmaf(du, yh, a_post[i][e]);
            }
            *reinterpret_cast<uint4 *>(p.dy + t * p.dy_stride + 8 * v) = pack8(dy);
            if (gate_tok && p.dgate)
                *reinterpret_cast<uint4 *>(p.dgate + t * p.dgate_stride + 8 * v) = pack8(dg);
        }
    }
    if (p.n_sum == 0) return;
    // the block's sums: its warps add theirs one after the other
    for (int w = 0; w < rows_per_block; ++w) {
        if (row_in_block == w) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = i * group + lane_in_row;
                if (v >= nvec) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float3 t = w > 0 ? s_sum[8 * v + e] : make_float3(0.f, 0.f, 0.f);
                    s_sum[8 * v + e] = make_float3(t.x + a_pre[i][e], t.y + a_post[i][e], t.z + a_gate[i][e]);
                }
            }
        }
        __syncthreads();
    }
    float *dst = p.part + (int64_t)blockIdx.x * p.n_sum * p.C;
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
        const float3 t = s_sum[c];
        if (p.at_pre >= 0) dst[(int64_t)p.at_pre * p.C + c] = t.x;
        if (p.at_post >= 0) dst[(int64_t)p.at_post * p.C + c] = t.y;
        if (p.at_gate >= 0) dst[(int64_t)p.at_gate * p.C + c] = t.z;
    }
}

// Rows above 512 columns: a block per row, fed by a ring of whole rows in shared memory, so that the
// loads in flight are the ring's and not the occupancy's: thread 0 keeps bulk copies of the block's
// next rows running while this one is reduced.
//
// One reduction (and one barrier) per row: dy needs sum_c A dH with A = scale gate w_post y, and
// dH = dh + r2 (a - h c2), a = dz w_pre, is linear in what the first reduction gives, so
//   sum A dH = sum A dh + r2 (sum A a - c2 sum A h)
// and six sums (h^2, a h, y^2, A dh, A a, A h) are taken at once.
// An input that a call does not have reads as zeros (or, for a gate, ones) from a part of shared memory
// filled once, and rows are padded with zeros to whole pieces of all lanes, so that the loops have no conditions.
struct Ring {
    int stages, slot;                          // slots, bytes of one
    int at_h, at_dz, at_dh, at_y, at_gate;     // byte offsets in slot 0
    int st_h, st_dz, st_dh, st_y, st_gate;     // and from slot to slot: `slot`, or 0 for what is filled once
    int fill, gate_fill;                       // the zeros' place, and that of a gate for all tokens (-1: none)
    int32_t *status;
};
constexpr int kMaxStages = 4;
constexpr long long kWaitBudget = 4000000000ll;   // clock cycles before a wait gives up (~2 s)

// Four consecutive values as two pairs for the packed fp32 instructions.
struct Quad {
    uint64_t a, b;
};
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Quad unpack4(const uint2 &a) {
    return {rope::f2(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u)),
            rope::f2(__uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u))};
}

// a piece (4 values) of a row in shared memory
template <bool F32> __device__ __forceinline__ Quad get4(const unsigned char *at) {
    if constexpr (F32) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(at);
        return {a.x, a.y};
    } else {
        return unpack4(*reinterpret_cast<const uint2 *>(at));
    }
}
// 4 consecutive values in bf16 or fp32
template <bool F32> __device__ __forceinline__ void put4(void *p, int64_t i, const Quad &x) {
    float v[4];
    rope::f2_split(x.a, v[0], v[1]);
    rope::f2_split(x.b, v[2], v[3]);
    if constexpr (F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + i) =
            make_uint2(rope::pack2(v[0], v[1]), rope::pack2(v[2], v[3]));
}

constexpr int kSums = 6;

// A lane holds NP pieces of 4 columns; its columns of the two weights stay in registers (from memory they
// come through an L1 that the ring leaves almost nothing of: 9001 x 5120 took 340 us that way). Measured at
// 9001 x 5120 with an fp32 residual and a gate per token: 168 us (6.0 TB/s); with two reductions per row
// 225 us. With conditions on what is there in the loops, 66 instead of about 30 instructions per column,
// 9001 x 5120 in bf16 took 162 instead of 144 us (125 with a constant number of threads).
// GROUP: the block's threads where they are a constant, and a lane's places with them (0: taken from the launch).
template <int NP, bool F32, int THREADS, int GROUP>
__global__ void __launch_bounds__(THREADS)
norm_residual_bwd_ring_kernel(const Bwd p, const Ring ring)
{
    using rope::f2_fma;
    using rope::f2_mul;
    constexpr int WARPS = THREADS / 32, RB = F32 ? 16 : 8;   // bytes of a piece of the residual stream
    extern __shared__ __align__(128) unsigned char s_ring[];
    __shared__ __align__(16) float s_red[2][WARPS][8];
    __shared__ uint64_t s_full[kMaxStages];
    const int never = 0;                       // no abort flag: every thread waits for itself
    grid_wait();
    grid_release();
    const int nvec = p.C >> 2, group = GROUP ? GROUP : (int)blockDim.x, wpr = group >> 5;
    const float inv_c = 1.f / (float)p.C;
    const bool gate_tok = p.gate && p.gate_stride != 0;
    const uint32_t row_b = 2u * (uint32_t)p.C, res_b = (F32 ? 4u : 2u) * (uint32_t)p.C;
    const uint32_t slot_b = (p.w_pre ? res_b + row_b : 0u) + (p.dh ? res_b : 0u) + (p.y ? row_b : 0u) +
                            (gate_tok ? row_b : 0u);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.stages; ++i) sm100::mbar_init(sm100::smem_addr(&s_full[i]), 1);
        sm100::fence_mbar_init();
    }
    // zeros everywhere that no copy writes
    for (int i = threadIdx.x; i < ring.stages * ring.slot / 16; i += blockDim.x)
        reinterpret_cast<uint4 *>(s_ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    const int padded = NP * group;             // pieces of a row
    for (int i = threadIdx.x; ring.fill >= 0 && i < padded; i += blockDim.x) {
        *reinterpret_cast<uint2 *>(s_ring + ring.fill + RB * i) = make_uint2(0u, 0u);
        if constexpr (F32) *reinterpret_cast<uint2 *>(s_ring + ring.fill + RB * i + 8) = make_uint2(0u, 0u);
    }
    constexpr uint32_t ONES = 0x3f803f80u;     // two bf16 1.0
    const auto weight_at = [&](const __nv_bfloat16 *w, int v, uint32_t none) {
        return !w || v >= nvec ? make_uint2(none, none) : *reinterpret_cast<const uint2 *>(w + 4 * v);
    };
    for (int i = threadIdx.x; ring.gate_fill >= 0 && i < padded; i += blockDim.x)
        *reinterpret_cast<uint2 *>(s_ring + ring.gate_fill + 8 * i) = weight_at(p.gate, i, ONES);
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // the copies come after these stores
    __syncthreads();
    const int n_rows = blockIdx.x < p.T ? (int)((p.T - 1 - blockIdx.x) / gridDim.x + 1) : 0;   // of this block
    auto fetch = [&](int k) {                  // thread 0: the block's k-th row into its slot
        const int64_t t = blockIdx.x + (int64_t)k * gridDim.x;
        const int s = k % ring.stages;
        const uint32_t bar = sm100::smem_addr(&s_full[s]);
        const uint32_t dst = sm100::smem_addr(s_ring) + s * ring.slot;   // (all that is copied is there per slot)
        sm100::mbar_arrive_expect_tx(bar, slot_b);
        const char *h = static_cast<const char *>(p.h), *dh = static_cast<const char *>(p.dh);
        if (p.w_pre) {
            sm100::bulk_load(dst + ring.at_h, h + t * p.h_stride * (F32 ? 4 : 2), res_b, bar);
            sm100::bulk_load(dst + ring.at_dz, p.dz + t * p.dz_stride, row_b, bar);
        }
        if (p.dh) sm100::bulk_load(dst + ring.at_dh, dh + t * p.dh_stride * (F32 ? 4 : 2), res_b, bar);
        if (p.y) sm100::bulk_load(dst + ring.at_y, p.y + t * p.y_stride, row_b, bar);
        if (gate_tok) sm100::bulk_load(dst + ring.at_gate, p.gate + t * p.gate_stride, row_b, bar);
    };
    int fetched = 0;
    if (threadIdx.x == 0)
        for (; fetched < n_rows && fetched < ring.stages; ++fetched) fetch(fetched);

    Quad a_pre[NP], a_post[NP], a_gate[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) a_pre[i] = a_post[i] = a_gate[i] = Quad{0ull, 0ull};
    Quad w_pre[NP], w_post[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int v = i * group + threadIdx.x;
        w_pre[i] = unpack4(weight_at(p.w_pre, v, 0u));
        w_post[i] = unpack4(weight_at(p.w_post, v, ONES));
    }
    struct Piece {
        Quad h, dh, dz, y, g;
    };
    const unsigned char *m_h = s_ring + ring.at_h + RB * threadIdx.x, *m_dh = s_ring + ring.at_dh + RB * threadIdx.x;
    const unsigned char *m_dz = s_ring + ring.at_dz + 8 * threadIdx.x, *m_y = s_ring + ring.at_y + 8 * threadIdx.x;
    const unsigned char *m_g = s_ring + ring.at_gate + 8 * threadIdx.x;
    auto values = [&](int s, int i, Piece &x) {
        x.h = get4<F32>(m_h + s * ring.st_h + i * RB * group);
        x.dh = get4<F32>(m_dh + s * ring.st_dh + i * RB * group);
        x.dz = get4<false>(m_dz + s * ring.st_dz + i * 8 * group);
        x.y = get4<false>(m_y + s * ring.st_y + i * 8 * group);
        x.g = get4<false>(m_g + s * ring.st_gate + i * 8 * group);
    };

    bool ok = true;
    int buf = 0, s_at = 0;
    uint32_t phase = 0;
    for (int k = 0; k < n_rows; ++k) {
        const int s = s_at;
        ok = __all_sync(0xffffffffu, sm100::mbar_wait(sm100::smem_addr(&s_full[s]), phase, &never, kWaitBudget));
        if (++s_at == ring.stages) {
            s_at = 0;
            phase ^= 1u;
        }
        if (ok) {
            uint64_t sum[kSums] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                Piece x;
                values(s, i, x);
                const Quad wr = w_pre[i], wo = w_post[i];
                auto add = [&](uint64_t h, uint64_t dh, uint64_t dz, uint64_t y, uint64_t g, uint64_t wr, uint64_t wo) {
                    const uint64_t a = f2_mul(dz, wr), A = f2_mul(f2_mul(g, wo), y);
                    sum[0] = f2_fma(h, h, sum[0]);
                    sum[1] = f2_fma(a, h, sum[1]);
                    sum[2] = f2_fma(y, y, sum[2]);
                    sum[3] = f2_fma(A, dh, sum[3]);
                    sum[4] = f2_fma(A, a, sum[4]);
                    sum[5] = f2_fma(A, h, sum[5]);
                };
                add(x.h.a, x.dh.a, x.dz.a, x.y.a, x.g.a, wr.a, wo.a);
                add(x.h.b, x.dh.b, x.dz.b, x.y.b, x.g.b, wr.b, wo.b);
            }
            float t[kSums];
#pragma unroll
            for (int j = 0; j < kSums; ++j) {
                float lo, hi;
                rope::f2_split(sum[j], lo, hi);
                t[j] = warp_sum(lo + hi);
            }
            if ((threadIdx.x & 31) == 0) {
                float *red = s_red[buf][threadIdx.x >> 5];
                *reinterpret_cast<float4 *>(red) = make_float4(t[0], t[1], t[2], t[3]);
                *reinterpret_cast<float2 *>(red + 4) = make_float2(t[4], t[5]);
            }
        }
        const auto *red = s_red[buf];
        buf ^= 1;
        ok = __syncthreads_and(ok);            // also agrees that the row has landed
        if (!ok) break;
        // every thread has left the row before
        if (threadIdx.x == 0 && k > 0 && fetched < n_rows) fetch(fetched++);
        const int64_t t = blockIdx.x + (int64_t)k * gridDim.x;
        float sum[kSums] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < wpr; ++w) {
            const float4 x = *reinterpret_cast<const float4 *>(red[w]);
            const float2 z = *reinterpret_cast<const float2 *>(red[w] + 4);
            sum[0] += x.x;
            sum[1] += x.y;
            sum[2] += x.z;
            sum[3] += x.w;
            sum[4] += z.x;
            sum[5] += z.y;
        }
        float r2 = 0.f, c2 = 0.f, r1 = 1.f, c1 = 0.f;
        if (p.w_pre) {
            r2 = rsqrtf(sum[0] * inv_c + p.eps);
            c2 = r2 * r2 * (sum[1] * inv_c);          // dH = dh + r2 (a - h c2)
        }
        if (p.w_post) {
            r1 = rsqrtf(sum[2] * inv_c + p.eps);
            c1 = r1 * r1 * (p.scale * fmaf(r2, fmaf(-c2, sum[5], sum[4]), sum[3]) * inv_c);   // dy = r1 (du w - y c1)
        }
        const uint64_t r2_2 = rope::f2(r2, r2), nc2 = rope::f2(-c2, -c2), r1_2 = rope::f2(r1, r1);
        const uint64_t nc1 = rope::f2(-c1, -c1), scale = rope::f2(p.scale, p.scale);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = i * group + threadIdx.x;
            Piece x;
            values(s, i, x);
            const Quad wr = w_pre[i], wo = w_post[i];
            Quad dx, dy, dg;
            auto back = [&](uint64_t h, uint64_t dh, uint64_t dz, uint64_t y, uint64_t g, uint64_t wr, uint64_t wo,
                            uint64_t &s_pre, uint64_t &s_post, uint64_t &s_gate, uint64_t &ox, uint64_t &oy,
                            uint64_t &og) {
                ox = f2_fma(r2_2, f2_fma(dz, wr, f2_mul(h, nc2)), dh);
                s_pre = f2_fma(dz, f2_mul(h, r2_2), s_pre);
                const uint64_t d = f2_mul(scale, ox), du = f2_mul(d, g), yh = f2_mul(y, r1_2);
                og = f2_mul(f2_mul(d, yh), wo);
                s_gate = f2_add(s_gate, og);
                s_post = f2_fma(du, yh, s_post);
                oy = p.w_post ? f2_mul(r1_2, f2_fma(du, wo, f2_mul(y, nc1))) : du;   // (0 y is not 0 for every y)
            };
            back(x.h.a, x.dh.a, x.dz.a, x.y.a, x.g.a, wr.a, wo.a, a_pre[i].a, a_post[i].a, a_gate[i].a, dx.a, dy.a,
                 dg.a);
            back(x.h.b, x.dh.b, x.dz.b, x.y.b, x.g.b, wr.b, wo.b, a_pre[i].b, a_post[i].b, a_gate[i].b, dx.b, dy.b,
                 dg.b);
            if (v >= nvec) continue;
            put4<F32>(p.dx, t * p.dx_stride + 4 * v, dx);
            put4<false>(p.dy, t * p.dy_stride + 4 * v, dy);
            if (gate_tok && p.dgate) put4<false>(p.dgate, t * p.dgate_stride + 4 * v, dg);
        }
    }
    if (!ok) {
        // a row never landed: say so, and let what was issued land before the shared memory goes
        if (threadIdx.x == 0) {
            report_error(ring.status, VIT_ERR_TIMEOUT);
            for (int k = fetched > ring.stages ? fetched - ring.stages : 0; k < fetched; ++k)
                sm100::mbar_wait(sm100::smem_addr(&s_full[k % ring.stages]), (uint32_t)(k / ring.stages) & 1, &never,
                                 20000000ll);
        }
        return;
    }
    if (p.n_sum == 0) return;
    float *dst = p.part + (int64_t)blockIdx.x * p.n_sum * p.C;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int v = i * group + threadIdx.x;
        if (v >= nvec) continue;
        if (p.at_pre >= 0) put4<true>(dst, (int64_t)p.at_pre * p.C + 4 * v, a_pre[i]);
        if (p.at_post >= 0) put4<true>(dst, (int64_t)p.at_post * p.C + 4 * v, a_post[i]);
        if (p.at_gate >= 0) put4<true>(dst, (int64_t)p.at_gate * p.C + 4 * v, a_gate[i]);
    }
}

// out_k[c] = sum over p of part[p][k][c], p in a fixed order: 32 columns a block, the partial rows
// dealt to 32 warps, their sums joined in warp order.
struct SumOut {
    float *out[3];
};
__global__ void __launch_bounds__(1024)
column_sum_kernel(const float *part, int n_parts, int n_sum, int C, const SumOut o)
{
    grid_wait();                               // the partial sums of the launch before
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t cols = (int64_t)n_sum * C;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float a = 0.f;
    if (col < cols)
        for (int q = warp; q < n_parts; q += 32) a += part[q * cols + col];
    s[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && col < cols) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 32; ++w) t += s[w][lane];
        o.out[col / C][col % C] = t;
    }
}

// Pieces of 8 columns per lane and warps per row. A row of one warp has no barriers; wider rows have as few
// warps as the registers allow. In bf16 that is one warp up to 6 pieces, then 4 pieces each (15000 x 4096: 82 us,
// 2 pieces 90, 1 piece 110; 6000 x 8192: 70, 82, 82). Pieces of an fp32 residual are twice as large: one warp
// up to 3 pieces, then 2 pieces each (60000 x 1024: 135 us, 4 pieces 164; 15000 x 4096: 141, 4 pieces 170, 1 piece
// 147).
void row_shape(int C, bool f32, int *vpt, int *wpr)
{
    const int nvec = C / 8, solo = f32 ? 3 : 6, each = f32 ? 2 : 4;
    *vpt = nvec <= 32 * solo ? (nvec + 31) / 32 : each;
    *wpr = (nvec + 32 * *vpt - 1) / (32 * *vpt);
}

template <int V> using Pieces = std::integral_constant<int, V>;

template <bool F32> cudaError_t launch_fwd(const Fwd &p, int num_sms, cudaStream_t stream)
{
    int vpt, wpr;
    row_shape(p.C, F32, &vpt, &wpr);
    const int rows = wpr == 1 ? 4 : 1;
    const int64_t want = (p.T + rows - 1) / rows, cap = (int64_t)num_sms * 64;
    const unsigned blocks = (unsigned)(want < cap ? want : cap);
    const int threads = 32 * wpr * rows;
    LaunchScope scope("norm_residual", stream);
    auto run = [&](auto v) {
        constexpr int V = decltype(v)::value;
        return launch_chained(wpr == 1 ? norm_residual_kernel<V, F32, true> : norm_residual_kernel<V, F32, false>, blocks,
                              threads, 0, stream, p, wpr, rows);
    };
    switch (vpt) {
        case 1: return run(Pieces<1>());
        case 2: return run(Pieces<2>());
        case 3: return run(Pieces<3>());
        default:
            if constexpr (!F32) {
                if (vpt == 4) return run(Pieces<4>());
                if (vpt == 5) return run(Pieces<5>());
                return run(Pieces<6>());
            }
            return cudaErrorInvalidValue;
    }
}

constexpr int kRingBytes = 224 * 1024;     // shared memory of an SM that the rings share
constexpr int kNarrow = 6144;              // widest row that 384 threads hold at four pieces each

// Pieces per lane and threads of a row's block. Fewer threads with more pieces each cost fewer shuffles and
// barriers per column (15000 x 4096 bf16: 225 us with two pieces and 512 threads, 185 with four and 256, before
// their number was a constant; 6000 x 8192: 220 us with six and 352, 109 with eight and 256). Eight below 6144 columns as well help where
// they fill the lanes (4096: 152 us) and not elsewhere (1280: 169 instead of 144 us, 520 with an fp32 residual
// 285 instead of 207). Threads of an SM: 384 (480, which the registers allow, leave each block too few slots:
// 37007 x 1280 with an fp32 residual 232 instead of 173 us; 320: 176).
int ring_threads(int C) { return C <= kNarrow ? (C / 4 + 127) / 128 * 32 : 256; }
// A constant number of threads is worth 10 to 14 % with a bf16 residual (15000 x 4096: 185 -> 160 us, 37007 x 1280: 143
// -> 127), where the loops are bound by their instructions, and nothing with an fp32 one; above 6144 columns
// the constants also keep eight pieces from spilling. A few numbers serve all widths.
int ring_threads_bf16(int C)
{
    const int t = ring_threads(C);
    return t <= 192 ? t : (t + 63) / 64 * 64;
}
int ring_blocks(int C) { return C <= kNarrow ? 384 / ring_threads(C) : 1; }

template <int NP, bool F32, int THREADS, int GROUP>
cudaError_t launch_ring(const Bwd &p, int32_t *status, int num_sms, unsigned *blocks, cudaStream_t stream)
{
    *blocks = 0;
    if (p.T == 0) return cudaSuccess;          // its tensors may be absent, all of them, and then a slot has no size
    const int threads = GROUP ? GROUP : ring_threads(p.C), cols = 4 * NP * threads;      // of a padded row
    const bool gate_tok = p.gate && p.gate_stride != 0;
    const int res_b = (F32 ? 4 : 2) * cols, row_b = 2 * cols;
    Ring r;
    r.status = status;
    r.slot = (p.w_pre ? res_b + row_b : 0) + (p.dh ? res_b : 0) + (p.y ? row_b : 0) + (gate_tok ? row_b : 0);
    const bool absent = !p.w_pre || !p.dh || !p.y;
    const int fixed = (absent ? res_b : 0) + (gate_tok ? 0 : row_b);
    // as many blocks per SM as its registers hold, each with two slots at least
    int ctas = THREADS / threads;
    while (ctas > 1 && kRingBytes / ctas < 2 * r.slot + fixed) --ctas;
    r.stages = (kRingBytes / ctas - fixed) / r.slot;
    if (r.stages > kMaxStages) r.stages = kMaxStages;
    if (r.stages < 2) return cudaErrorInvalidValue;
    r.fill = absent ? r.stages * r.slot : -1;
    r.gate_fill = gate_tok ? -1 : r.stages * r.slot + (absent ? res_b : 0);
    int at = 0;
    auto place = [&](bool there, int bytes, int &where, int &step) {
        where = there ? at : r.fill;
        step = there ? r.slot : 0;
        if (there) at += bytes;
    };
    place(p.w_pre != nullptr, res_b, r.at_h, r.st_h);
    place(p.w_pre != nullptr, row_b, r.at_dz, r.st_dz);
    place(p.dh != nullptr, res_b, r.at_dh, r.st_dh);
    place(p.y != nullptr, row_b, r.at_y, r.st_y);
    place(gate_tok, row_b, r.at_gate, r.st_gate);
    if (!gate_tok) r.at_gate = r.gate_fill;
    int64_t most = (int64_t)num_sms * ctas;
    if (most > norm_residual_parts(p.C)) most = norm_residual_parts(p.C);
    *blocks = (unsigned)(p.T < most ? p.T : most);
    auto kern = norm_residual_bwd_ring_kernel<NP, F32, THREADS, GROUP>;
    static DeviceOnce once;
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    });
    if (e != cudaSuccess) return e;
    LaunchScope scope("norm_residual_bwd", stream);
    return launch_chained(kern, *blocks, threads, (size_t)r.stages * r.slot + fixed, stream, p, r);
}

template <bool F32>
cudaError_t launch_bwd(const Bwd &p, const SumOut &o, int32_t *status, int num_sms, cudaStream_t stream)
{
    unsigned blocks = 0;
    cudaError_t e = cudaSuccess;
    if (p.C <= 512) {
        const int rows = 8;
        const int64_t want = (p.T + rows - 1) / rows;
        const int64_t most = (int64_t)num_sms * 4, parts = norm_residual_parts(p.C), cap = most < parts ? most : parts;
        blocks = (unsigned)(want < cap ? want : cap);
        if (blocks > 0) {
            LaunchScope scope("norm_residual_bwd", stream);
            e = launch_chained(p.C <= 256 ? norm_residual_bwd_kernel<1, F32> : norm_residual_bwd_kernel<2, F32>, blocks,
                               32 * rows, 0, stream, p, rows);
        }
    } else if (p.C > kNarrow) {
        e = launch_ring<8, F32, 256, 256>(p, status, num_sms, &blocks, stream);
    } else if constexpr (F32) {
        e = launch_ring<4, F32, 384, 0>(p, status, num_sms, &blocks, stream);
    } else {
        switch (ring_threads_bf16(p.C)) {
            case 64: e = launch_ring<4, F32, 384, 64>(p, status, num_sms, &blocks, stream); break;
            case 96: e = launch_ring<4, F32, 384, 96>(p, status, num_sms, &blocks, stream); break;
            case 128: e = launch_ring<4, F32, 384, 128>(p, status, num_sms, &blocks, stream); break;
            case 160: e = launch_ring<4, F32, 384, 160>(p, status, num_sms, &blocks, stream); break;
            case 192: e = launch_ring<4, F32, 384, 192>(p, status, num_sms, &blocks, stream); break;
            case 256: e = launch_ring<4, F32, 384, 256>(p, status, num_sms, &blocks, stream); break;
            case 320: e = launch_ring<4, F32, 384, 320>(p, status, num_sms, &blocks, stream); break;
            default: e = launch_ring<4, F32, 384, 384>(p, status, num_sms, &blocks, stream); break;
        }
    }
    if (e != cudaSuccess || p.n_sum == 0) return e;
    return launch_column_sum(p.part, (int)blocks, p.n_sum, p.C, o.out[0], o.out[1], o.out[2], stream);
}

}  // namespace

// Blocks of the gradient kernel at most, each of which leaves a row of sums.
int norm_residual_parts(int C) { return kDesignSms * (C <= 512 ? 4 : ring_blocks(C)); }

cudaError_t launch_column_sum(const float *part, int n_parts, int n_sum, int C, float *out0, float *out1, float *out2,
                              cudaStream_t stream)
{
    const SumOut o{{out0, out1, out2}};
    LaunchScope scope("column_sum", stream);
    return launch_chained(column_sum_kernel, (unsigned)(((int64_t)n_sum * C + 31) / 32), 1024, 0, stream, part, n_parts,
                          n_sum, C, o);
}

cudaError_t launch_norm_residual(const NormResidualArgs &a, int num_sms, cudaStream_t stream)
{
    Fwd p;
    p.x = a.x;
    p.y = static_cast<const __nv_bfloat16 *>(a.y);
    p.gate = static_cast<const __nv_bfloat16 *>(a.gate);
    p.w_post = static_cast<const __nv_bfloat16 *>(a.w_post);
    p.w_pre = static_cast<const __nv_bfloat16 *>(a.w_pre);
    p.h = a.h_out;
    p.z = static_cast<__nv_bfloat16 *>(a.z_out);
    p.T = a.T;
    p.x_stride = a.x_stride;
    p.y_stride = a.y_stride;
    p.gate_stride = a.gate_stride;
    p.h_stride = a.h_stride;
    p.z_stride = a.z_stride;
    p.C = a.C;
    p.scale = a.scale;
    p.eps = a.eps;
    return a.res_f32 ? launch_fwd<true>(p, num_sms, stream) : launch_fwd<false>(p, num_sms, stream);
}

cudaError_t launch_norm_residual_bwd(const NormResidualGrad &a, int num_sms, cudaStream_t stream)
{
    Bwd p;
    p.dz = static_cast<const __nv_bfloat16 *>(a.dz);
    p.dh = a.dh;
    p.h = a.h;
    p.y = static_cast<const __nv_bfloat16 *>(a.y);
    p.gate = static_cast<const __nv_bfloat16 *>(a.gate);
    p.w_post = static_cast<const __nv_bfloat16 *>(a.w_post);
    p.w_pre = static_cast<const __nv_bfloat16 *>(a.w_pre);
    p.dx = a.dx;
    p.dy = static_cast<__nv_bfloat16 *>(a.dy);
    const bool gate_tok = a.gate && a.gate_stride != 0;
    p.dgate = gate_tok ? static_cast<__nv_bfloat16 *>(a.dgate) : nullptr;
    p.part = a.part;
    p.T = a.T;
    p.dz_stride = a.dz_stride;
    p.dh_stride = a.dh_stride;
    p.h_stride = a.h_stride;
    p.y_stride = a.y_stride;
    p.gate_stride = a.gate_stride;
    p.dx_stride = a.dx_stride;
    p.dy_stride = a.dy_stride;
    p.dgate_stride = a.dgate_stride;
    p.C = a.C;
    p.scale = a.scale;
    p.eps = a.eps;
    SumOut o{{nullptr, nullptr, nullptr}};
    p.n_sum = 0;
    auto place = [&](bool asked, float *out) {
        if (!asked) return -1;
        o.out[p.n_sum] = out;
        return p.n_sum++;
    };
    p.at_pre = place(a.dw_pre != nullptr, a.dw_pre);
    p.at_post = place(a.dw_post != nullptr, a.dw_post);
    p.at_gate = place(a.gate && !gate_tok && a.dgate, static_cast<float *>(a.dgate));
    return a.res_f32 ? launch_bwd<true>(p, o, a.status, num_sms, stream) : launch_bwd<false>(p, o, a.status, num_sms, stream);
}

}  // namespace vit
