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
// Everything is HBM bound: a row is read once into registers, both reductions run on it there in
// fp32, and it is written once. A row belongs to a group of `wpr` warps, each lane holding VPT
// pieces of 8 columns; a group of one warp needs shuffles only, larger ones (a whole block) meet
// in shared memory. h is normalised before it is rounded to its storage type; the gradient
// recomputes r2 from the stored h it is given.
//
// The sums over tokens are accumulated in registers by persistent groups (a lane keeps its columns
// from row to row), written once per group as a partial row of the workspace and added up by a
// second small kernel in a fixed order, so results do not change from run to run.
#include "internal.h"
#include "rope_math.cuh"
#include "sm100.cuh"

namespace vit {
namespace {

constexpr int kMaxWarps = 16;             // per row: rows of up to 8192 columns with two pieces per lane

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

template <int VPT, bool F32>
__global__ void __launch_bounds__(512)
norm_residual_kernel(const Fwd p, int wpr, int rows_per_block)
{
    __shared__ float s_red[2 * kMaxWarps];
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
struct Ring {
    int stages, slot;                          // slots, bytes of one
    int at_dz, at_dh, at_y, at_gate;           // byte offsets in a slot (h is at 0)
    int32_t *status;
};
constexpr int kMaxStages = 4;
constexpr long long kWaitBudget = 4000000000ll;   // clock cycles before a wait gives up (~2 s)

__device__ __forceinline__ void unpack4(const uint2 &a, float *x) {
    x[0] = __uint_as_float(a.x << 16);
    x[1] = __uint_as_float(a.x & 0xffff0000u);
    x[2] = __uint_as_float(a.y << 16);
    x[3] = __uint_as_float(a.y & 0xffff0000u);
}

// piece v (4 values) of a row in shared memory, or 0
template <bool F32> __device__ __forceinline__ void get4(bool there, const unsigned char *row, int v, float *x) {
    if constexpr (F32) {
        const float4 a = there ? *reinterpret_cast<const float4 *>(row + 16 * v) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    } else {
        unpack4(there ? *reinterpret_cast<const uint2 *>(row + 8 * v) : make_uint2(0u, 0u), x);
    }
}
// 4 consecutive values in bf16 or fp32
template <bool F32> __device__ __forceinline__ void put4(void *p, int64_t i, const float *x) {
    if constexpr (F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + i) =
            make_uint2(rope::pack2(x[0], x[1]), rope::pack2(x[2], x[3]));
}

constexpr int kSums = 6;

// keeps the loads of a lane's pieces (4 columns each, so that few values are live beside the sums) apart
__device__ __forceinline__ void one_piece() { asm volatile("" ::: "memory"); }

// WR: the lane's columns of the weights and of a gate of all tokens stay in registers (from memory
// they come through an L1 that the ring leaves almost nothing of: 9001 x 5120 took 340 us that way).
// Rows above 5120 columns, six pieces per lane, have no room for them. Measured at 9001 x 5120 with an
// fp32 residual and a gate per token: 176 us (5.76 TB/s); with two reductions per row 225 us; with the
// row's values kept in registers as well 275 us; with two pieces per lane and 640 threads 180 us.
template <int NP, bool F32, bool WR>
__global__ void __launch_bounds__(NP == 2 ? 512 : NP == 4 ? 320 : 352)
norm_residual_bwd_ring_kernel(const Bwd p, const Ring ring)
{
    extern __shared__ __align__(128) unsigned char s_ring[];
    __shared__ __align__(16) float s_red[2][kMaxWarps][8];
    __shared__ uint64_t s_full[kMaxStages];
    const int never = 0;                       // no abort flag: every thread waits for itself
    grid_release();
    const int nvec = p.C >> 2, group = blockDim.x, wpr = blockDim.x >> 5;
    const float inv_c = 1.f / (float)p.C;
    const bool gate_tok = p.gate && p.gate_stride != 0;
    const uint32_t row_b = 2u * (uint32_t)p.C, res_b = (F32 ? 4u : 2u) * (uint32_t)p.C;
    const uint32_t slot_b = (p.w_pre ? res_b + row_b : 0u) + (p.dh ? res_b : 0u) + (p.y ? row_b : 0u) +
                            (gate_tok ? row_b : 0u);
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.stages; ++i) sm100::mbar_init(sm100::smem_addr(&s_full[i]), 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    const int n_rows = blockIdx.x < p.T ? (int)((p.T - 1 - blockIdx.x) / gridDim.x + 1) : 0;   // of this block
    auto fetch = [&](int k) {                  // thread 0: the block's k-th row into its slot
        const int64_t t = blockIdx.x + (int64_t)k * gridDim.x;
        const int s = k % ring.stages;
        const uint32_t bar = sm100::smem_addr(&s_full[s]);
        const uint32_t dst = sm100::smem_addr(s_ring) + s * ring.slot;
        sm100::mbar_arrive_expect_tx(bar, slot_b);
        const char *h = static_cast<const char *>(p.h), *dh = static_cast<const char *>(p.dh);
        if (p.w_pre) {
            sm100::bulk_load(dst, h + t * p.h_stride * (F32 ? 4 : 2), res_b, bar);
            sm100::bulk_load(dst + ring.at_dz, p.dz + t * p.dz_stride, row_b, bar);
        }
        if (p.dh) sm100::bulk_load(dst + ring.at_dh, dh + t * p.dh_stride * (F32 ? 4 : 2), res_b, bar);
        if (p.y) sm100::bulk_load(dst + ring.at_y, p.y + t * p.y_stride, row_b, bar);
        if (gate_tok) sm100::bulk_load(dst + ring.at_gate, p.gate + t * p.gate_stride, row_b, bar);
    };
    int fetched = 0;
    if (threadIdx.x == 0)
        for (; fetched < n_rows && fetched < ring.stages; ++fetched) fetch(fetched);

    float a_pre[NP][4], a_post[NP][4], a_gate[NP][4];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) a_pre[i][e] = a_post[i][e] = a_gate[i][e] = 0.f;
    constexpr int NH = WR ? NP : 1;
    uint2 r_pre[NH], r_post[NH], r_gate[NH];
    if constexpr (WR) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = i * group + threadIdx.x;
            const auto take = [&](const __nv_bfloat16 *w) {
                return w && v < nvec ? *reinterpret_cast<const uint2 *>(w + 4 * v) : make_uint2(0u, 0u);
            };
            r_pre[i] = take(p.w_pre);
            r_post[i] = take(p.w_post);
            r_gate[i] = take(gate_tok ? nullptr : p.gate);
        }
    }
    // one piece of a row: 0 where an input is not there, 1 for a missing gate or post-norm weight
    struct Piece {
        float h[4], dh[4], dz[4], y[4], g[4], wr[4], wo[4];
    };
    auto values = [&](const unsigned char *slot, int i, Piece &x) {
        const int v = i * group + threadIdx.x, k = WR ? i : 0;
        const bool in = v < nvec;
        auto word = [&](bool there, int at) {
            return there && in ? *reinterpret_cast<const uint2 *>(slot + at + 8 * v) : make_uint2(0u, 0u);
        };
        get4<F32>(p.w_pre && in, slot, v, x.h);
        get4<F32>(p.dh && in, slot + ring.at_dh, v, x.dh);
        unpack4(word(p.w_pre, ring.at_dz), x.dz);
        unpack4(word(p.y, ring.at_y), x.y);
        auto weight = [&](const __nv_bfloat16 *w, const uint2 &reg, float *o) {
            if constexpr (WR)
                unpack4(reg, o);
            else
                unpack4(w && in ? *reinterpret_cast<const uint2 *>(w + 4 * v) : make_uint2(0u, 0u), o);
        };
        weight(p.w_pre, r_pre[k], x.wr);
        if (gate_tok)
            unpack4(word(true, ring.at_gate), x.g);
        else if (p.gate)
            weight(p.gate, r_gate[k], x.g);
        if (p.w_post) weight(p.w_post, r_post[k], x.wo);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!p.gate) x.g[e] = 1.f;
            if (!p.w_post) x.wo[e] = 1.f;
        }
    };

    bool ok = true;
    int s_at = 0, buf = 0;
    uint32_t phase = 0;
    for (int k = 0; k < n_rows; ++k) {
        const int64_t t = blockIdx.x + (int64_t)k * gridDim.x;
        const unsigned char *slot = s_ring + s_at * ring.slot;
        ok = __all_sync(0xffffffffu, sm100::mbar_wait(sm100::smem_addr(&s_full[s_at]), phase, &never, kWaitBudget));
        if (++s_at == ring.stages) {
            s_at = 0;
            phase ^= 1u;
        }
        float sum[kSums] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (ok) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if constexpr (!WR) one_piece();
                Piece x;
                values(slot, i, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = x.dz[e] * x.wr[e], A = x.g[e] * x.wo[e] * x.y[e];
                    sum[0] = fmaf(x.h[e], x.h[e], sum[0]);
                    sum[1] = fmaf(a, x.h[e], sum[1]);
                    sum[2] = fmaf(x.y[e], x.y[e], sum[2]);
                    sum[3] = fmaf(A, x.dh[e], sum[3]);
                    sum[4] = fmaf(A, a, sum[4]);
                    sum[5] = fmaf(A, x.h[e], sum[5]);
                }
            }
#pragma unroll
            for (int j = 0; j < kSums; ++j) sum[j] = warp_sum(sum[j]);
        }
        float(*red)[8] = s_red[buf];
        buf ^= 1;
        if ((threadIdx.x & 31) == 0) {
            *reinterpret_cast<float4 *>(red[threadIdx.x >> 5]) = make_float4(sum[0], sum[1], sum[2], sum[3]);
            *reinterpret_cast<float2 *>(red[threadIdx.x >> 5] + 4) = make_float2(sum[4], sum[5]);
        }
        ok = __syncthreads_and(ok);            // also agrees that the row has landed
        if (!ok) break;
        // every thread has left the row before
        if (threadIdx.x == 0 && k > 0 && fetched < n_rows) fetch(fetched++);
#pragma unroll
        for (int j = 0; j < kSums; ++j) sum[j] = 0.f;
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
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = i * group + threadIdx.x;
            if constexpr (!WR) one_piece();
            if (v >= nvec) continue;
            Piece x;
            values(slot, i, x);
            float dx[4], dy[4], dg[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dx[e] = fmaf(r2, fmaf(x.dz[e], x.wr[e], -x.h[e] * c2), x.dh[e]);
                a_pre[i][e] = fmaf(x.dz[e], x.h[e] * r2, a_pre[i][e]);
                const float d = p.scale * dx[e], du = d * x.g[e], yh = x.y[e] * r1;
                dg[e] = d * yh * x.wo[e];
                a_gate[i][e] += dg[e];
                a_post[i][e] = fmaf(du, yh, a_post[i][e]);
                dy[e] = p.w_post ? r1 * fmaf(du, x.wo[e], -x.y[e] * c1) : du;
            }
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
column_sum_kernel(const float *__restrict__ part, int n_parts, int n_sum, int C, const SumOut o)
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

// Columns per lane and warps per row: the fewest pieces per lane with which a row fits `max_warps`
// warps; a row of one warp is preferred up to `solo` pieces per lane (no barriers).
void row_shape(int C, int solo, int max_vpt, int max_warps, int *vpt, int *wpr)
{
    const int nvec = C / 8;
    if (nvec <= 32 * solo) {
        *wpr = 1;
        *vpt = (nvec + 31) / 32;
        return;
    }
    for (int v = 1; v <= max_vpt; ++v) {
        const int w = (nvec + 32 * v - 1) / (32 * v);
        if (w <= max_warps) {
            *vpt = v;
            *wpr = w;
            return;
        }
    }
    *vpt = max_vpt;
    *wpr = (nvec + 32 * max_vpt - 1) / (32 * max_vpt);
}

template <bool F32> cudaError_t launch_fwd(const Fwd &p, int num_sms, cudaStream_t stream)
{
    int vpt, wpr;
    row_shape(p.C, 6, 4, 16, &vpt, &wpr);
    const int rows = wpr == 1 ? 4 : 1;
    const int64_t want = (p.T + rows - 1) / rows, cap = (int64_t)num_sms * 64;
    const unsigned blocks = (unsigned)(want < cap ? want : cap);
    const int threads = 32 * wpr * rows;
    LaunchScope scope("norm_residual", stream);
    switch (vpt) {
        case 1: norm_residual_kernel<1, F32><<<blocks, threads, 0, stream>>>(p, wpr, rows); break;
        case 2: norm_residual_kernel<2, F32><<<blocks, threads, 0, stream>>>(p, wpr, rows); break;
        case 3: norm_residual_kernel<3, F32><<<blocks, threads, 0, stream>>>(p, wpr, rows); break;
        case 4: norm_residual_kernel<4, F32><<<blocks, threads, 0, stream>>>(p, wpr, rows); break;
        case 5: norm_residual_kernel<5, F32><<<blocks, threads, 0, stream>>>(p, wpr, rows); break;
        case 6: norm_residual_kernel<6, F32><<<blocks, threads, 0, stream>>>(p, wpr, rows); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

constexpr int kRingBytes = 224 * 1024;     // shared memory of an SM that the rings share

template <int NP, bool F32, bool WR>
cudaError_t launch_ring(const Bwd &p, int32_t *status, int num_sms, unsigned *blocks, cudaStream_t stream)
{
    const int res_b = (F32 ? 4 : 2) * p.C, row_b = 2 * p.C;
    Ring r;
    int at = p.w_pre ? res_b : 0;
    auto place = [&](bool there, int bytes) {
        const int here = at;
        if (there) at += bytes;
        return here;
    };
    r.at_dz = place(p.w_pre != nullptr, row_b);
    r.at_dh = place(p.dh != nullptr, res_b);
    r.at_y = place(p.y != nullptr, row_b);
    r.at_gate = place(p.gate && p.gate_stride != 0, row_b);
    r.slot = (at + 127) / 128 * 128;
    r.status = status;
    const int threads = (p.C / 4 + 32 * NP - 1) / (32 * NP) * 32;
    // as many blocks per SM as its registers hold, each with two slots at least
    int ctas = 512 / threads;
    while (ctas > 1 && kRingBytes / ctas < 2 * r.slot) --ctas;
    r.stages = kRingBytes / ctas / r.slot;
    if (r.stages > kMaxStages) r.stages = kMaxStages;
    if (r.stages < 2) return cudaErrorInvalidValue;
    int64_t most = (int64_t)num_sms * ctas;
    if (most > kNormResidualParts) most = kNormResidualParts;
    *blocks = (unsigned)(p.T < most ? p.T : most);
    if (*blocks == 0) return cudaSuccess;
    auto kern = norm_residual_bwd_ring_kernel<NP, F32, WR>;
    static DeviceOnce once;
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    });
    if (e != cudaSuccess) return e;
    LaunchScope scope("norm_residual_bwd", stream);
    kern<<<*blocks, threads, (size_t)r.stages * r.slot, stream>>>(p, r);
    return cudaGetLastError();
}

template <bool F32>
cudaError_t launch_bwd(const Bwd &p, const SumOut &o, int32_t *status, int num_sms, cudaStream_t stream)
{
    unsigned blocks = 0;
    cudaError_t e = cudaSuccess;
    if (p.C <= 512) {
        const int rows = 8;
        const int64_t want = (p.T + rows - 1) / rows;
        const int64_t most = (int64_t)num_sms * 4, cap = most < kNormResidualParts ? most : kNormResidualParts;
        blocks = (unsigned)(want < cap ? want : cap);
        if (blocks > 0) {
            LaunchScope scope("norm_residual_bwd", stream);
            if (p.C <= 256) norm_residual_bwd_kernel<1, F32><<<blocks, 32 * rows, 0, stream>>>(p, rows);
            else norm_residual_bwd_kernel<2, F32><<<blocks, 32 * rows, 0, stream>>>(p, rows);
            e = cudaGetLastError();
        }
    } else if (p.C <= 4096) {
        e = launch_ring<2, F32, true>(p, status, num_sms, &blocks, stream);
    } else if (p.C <= 5120) {
        e = launch_ring<4, F32, true>(p, status, num_sms, &blocks, stream);
    } else {
        e = launch_ring<6, F32, false>(p, status, num_sms, &blocks, stream);
    }
    if (e != cudaSuccess || p.n_sum == 0) return e;
    return launch_column_sum(p.part, (int)blocks, p.n_sum, p.C, o.out[0], o.out[1], o.out[2], stream);
}

}  // namespace

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
