// C ABI of the operators around a language model's reading of the encoder's states: argument
// validation on the host, then kernel launches (as in api.cu).
#include <math.h>

#include "cross.h"
#include "internal.h"
#include "trace.h"

using namespace vit;

namespace {

bool head_dim_ok(int D) { return D == 32 || D == 64 || D == 80 || D == 96 || D == 128; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool stride_ok(int64_t s, int64_t n) { return s >= n && s % 8 == 0; }
bool heads_ok(int H) { return H >= 1 && H <= 65536; }
vit_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? VIT_OK : VIT_ERR_CUDA; }

constexpr int64_t kMaxTokens = (int64_t)1 << 31;
constexpr int64_t kMaxRows = kMaxTokens - (1 << 16);   // of a cross-attention side: a tile past the end still fits an int
constexpr int kMaxWidth = 8192;

// the checks that the three-axis rotary calls share
vit_status_t check_mrope(int64_t T, bool has_q, bool has_k, int Hq, int Hk, int D, const int32_t *pos,
                         const float *inv_freq, const int *sections, int axis_layout, int rope_mode,
                         const void *norm_w, float eps)
{
    if (!head_dim_ok(D)) return VIT_ERR_BAD_HEAD_DIM;
    if (T < 0 || T >= kMaxTokens || (has_q && !heads_ok(Hq)) || (has_k && !heads_ok(Hk))) return VIT_ERR_BAD_SHAPE;
    if (!(eps >= 0.f) || !isfinite(eps)) return VIT_ERR_BAD_ARGUMENT;
    if (rope_mode != VIT_ROPE_ROTATE_HALF && rope_mode != VIT_ROPE_INTERLEAVED) return VIT_ERR_BAD_ARGUMENT;
    if (axis_layout != VIT_MROPE_BLOCKED && axis_layout != VIT_MROPE_CYCLED) return VIT_ERR_BAD_ARGUMENT;
    if (!sections) return VIT_ERR_NULL_POINTER;
    for (int a = 0; a < 3; ++a)
        if (sections[a] < 0 || sections[a] > D / 2) return VIT_ERR_BAD_ARGUMENT;
    if (sections[0] + sections[1] + sections[2] != D / 2) return VIT_ERR_BAD_ARGUMENT;
    if (axis_layout == VIT_MROPE_CYCLED && (3 * sections[1] > D / 2 + 1 || 3 * sections[2] > D / 2))
        return VIT_ERR_BAD_ARGUMENT;
    if (T > 0 && ((!has_q && !has_k) || !pos || !inv_freq)) return VIT_ERR_NULL_POINTER;
    if (((uintptr_t)pos & 3u) || ((uintptr_t)inv_freq & 3u) || !aligned16(norm_w)) return VIT_ERR_MISALIGNED;
    return VIT_OK;
}

}  // namespace

extern "C" {

vit_status_t vit_grid_positions(const int32_t *grid_thw, int n, int64_t T, int32_t *pos_thw, int32_t *cu_seqlens,
                                int32_t *status_dev, vit_stream_t stream)
{
    TraceRange trace("vit_grid_positions");
    if (n < 0 || T < 0 || T >= kMaxTokens) return VIT_ERR_BAD_SHAPE;
    if (n > VIT_MAX_SEGMENTS) return VIT_ERR_TOO_MANY_SEGMENTS;
    if (n > 0 && !grid_thw) return VIT_ERR_NULL_POINTER;
    if (((uintptr_t)grid_thw & 3u) || ((uintptr_t)pos_thw & 3u) || ((uintptr_t)cu_seqlens & 3u))
        return VIT_ERR_MISALIGNED;
    if (!pos_thw && !cu_seqlens) return VIT_OK;
    int sms = 0;
    vit_status_t st = check_device(&sms);
    if (st != VIT_OK) return st;
    return from_cuda(launch_grid_positions(grid_thw, n, T, pos_thw, cu_seqlens, status_dev, sms, (cudaStream_t)stream));
}

vit_status_t vit_qk_norm_mrope(const void *q_in, void *q_out, const void *k_in, void *k_out, int64_t T, int Hq, int Hk,
                               int D, int64_t q_in_stride, int64_t q_out_stride, int64_t k_in_stride,
                               int64_t k_out_stride, const int32_t *pos_thw, const float *inv_freq,
                               const int *sections, int axis_layout, int rope_mode, const void *norm_w, float eps,
                               vit_stream_t stream)
{
    TraceRange trace("vit_qk_norm_mrope");
    const bool has_q = q_in || q_out, has_k = k_in || k_out;
    vit_status_t st = check_mrope(T, has_q, has_k, Hq, Hk, D, pos_thw, inv_freq, sections, axis_layout, rope_mode,
                                  norm_w, eps);
    if (st != VIT_OK) return st;
    if (T == 0) return VIT_OK;
    if ((has_q && (!q_in || !q_out)) || (has_k && (!k_in || !k_out))) return VIT_ERR_NULL_POINTER;
    if (has_q && (!stride_ok(q_in_stride, (int64_t)Hq * D) || !stride_ok(q_out_stride, (int64_t)Hq * D) ||
                  (q_in == q_out && q_in_stride != q_out_stride)))
        return VIT_ERR_BAD_STRIDE;
    if (has_k && (!stride_ok(k_in_stride, (int64_t)Hk * D) || !stride_ok(k_out_stride, (int64_t)Hk * D) ||
                  (k_in == k_out && k_in_stride != k_out_stride)))
        return VIT_ERR_BAD_STRIDE;
    if (!aligned16(q_in) || !aligned16(q_out) || !aligned16(k_in) || !aligned16(k_out)) return VIT_ERR_MISALIGNED;
    int sms = 0;
    st = check_device(&sms);
    if (st != VIT_OK) return st;
    MropeArgs a{};
    a.q_in = q_in;
    a.q_out = q_out;
    a.k_in = k_in;
    a.k_out = k_out;
    a.q_in_stride = q_in_stride;
    a.q_out_stride = q_out_stride;
    a.k_in_stride = k_in_stride;
    a.k_out_stride = k_out_stride;
    a.T = T;
    a.Hq = has_q ? Hq : 0;
    a.Hk = has_k ? Hk : 0;
    a.D = D;
    a.pos = pos_thw;
    a.inv_freq = inv_freq;
    for (int i = 0; i < 3; ++i) a.sections[i] = sections[i];
    a.cycled = axis_layout == VIT_MROPE_CYCLED;
    a.interleaved = rope_mode == VIT_ROPE_INTERLEAVED;
    a.norm_w = norm_w;
    a.eps = eps;
    return from_cuda(launch_mrope(a, sms, (cudaStream_t)stream));
}

size_t vit_qk_norm_mrope_bwd_workspace_size(int D)
{
    return head_dim_ok(D) ? sizeof(float) * 2 * (size_t)D * kMropeParts : 0;
}

vit_status_t vit_qk_norm_mrope_bwd(const void *dq_out, void *dq_in, const void *dk_out, void *dk_in, const void *q_in,
                                   const void *k_in, int64_t T, int Hq, int Hk, int D, int64_t dq_out_stride,
                                   int64_t dq_in_stride, int64_t dk_out_stride, int64_t dk_in_stride,
                                   int64_t q_in_stride, int64_t k_in_stride, const int32_t *pos_thw,
                                   const float *inv_freq, const int *sections, int axis_layout, int rope_mode,
                                   const void *norm_w, float eps, float *dnorm_w, void *workspace,
                                   size_t workspace_bytes, vit_stream_t stream)
{
    TraceRange trace("vit_qk_norm_mrope_bwd");
    const bool has_q = dq_out || dq_in, has_k = dk_out || dk_in;
    vit_status_t st = check_mrope(T, has_q, has_k, Hq, Hk, D, pos_thw, inv_freq, sections, axis_layout, rope_mode,
                                  norm_w, eps);
    if (st != VIT_OK) return st;
    if (!norm_w) dnorm_w = nullptr;
    if (T == 0 && !dnorm_w) return VIT_OK;
    if (T > 0) {
        if ((has_q && (!dq_out || !dq_in || (norm_w && !q_in))) || (has_k && (!dk_out || !dk_in || (norm_w && !k_in))))
            return VIT_ERR_NULL_POINTER;
        const int64_t nq = (int64_t)Hq * D, nk = (int64_t)Hk * D;
        if (has_q && (!stride_ok(dq_out_stride, nq) || !stride_ok(dq_in_stride, nq) ||
                      (norm_w && !stride_ok(q_in_stride, nq)) || (dq_out == dq_in && dq_out_stride != dq_in_stride)))
            return VIT_ERR_BAD_STRIDE;
        if (has_k && (!stride_ok(dk_out_stride, nk) || !stride_ok(dk_in_stride, nk) ||
                      (norm_w && !stride_ok(k_in_stride, nk)) || (dk_out == dk_in && dk_out_stride != dk_in_stride)))
            return VIT_ERR_BAD_STRIDE;
        if (!aligned16(dq_out) || !aligned16(dq_in) || !aligned16(dk_out) || !aligned16(dk_in) ||
            (norm_w && (!aligned16(q_in) || !aligned16(k_in))))
            return VIT_ERR_MISALIGNED;
    }
    if (dnorm_w) {
        if (!workspace) return VIT_ERR_NULL_POINTER;
        if (((uintptr_t)dnorm_w & 3u) || !aligned16(workspace)) return VIT_ERR_MISALIGNED;
        if (workspace_bytes < vit_qk_norm_mrope_bwd_workspace_size(D)) return VIT_ERR_WORKSPACE_TOO_SMALL;
    }
    int sms = 0;
    st = check_device(&sms);
    if (st != VIT_OK) return st;
    MropeArgs a{};
    a.q_in = q_in;
    a.k_in = k_in;
    a.q_out = dq_in;
    a.k_out = dk_in;
    a.dq = dq_out;
    a.dk = dk_out;
    a.q_in_stride = q_in_stride;
    a.k_in_stride = k_in_stride;
    a.q_out_stride = dq_in_stride;
    a.k_out_stride = dk_in_stride;
    a.dq_stride = dq_out_stride;
    a.dk_stride = dk_out_stride;
    a.T = T;
    a.Hq = has_q ? Hq : 0;
    a.Hk = has_k ? Hk : 0;
    a.D = D;
    a.pos = pos_thw;
    a.inv_freq = inv_freq;
    for (int i = 0; i < 3; ++i) a.sections[i] = sections[i];
    a.cycled = axis_layout == VIT_MROPE_CYCLED;
    a.interleaved = rope_mode == VIT_ROPE_INTERLEAVED;
    a.norm_w = norm_w;
    a.eps = eps;
    a.part = static_cast<float *>(workspace);
    return from_cuda(launch_mrope_bwd(a, dnorm_w, sms, (cudaStream_t)stream));
}

namespace {

// bounds of the lengths as the kernels take them, and whether the sizes of a cross-attention call fit
vit_status_t cross_sizes(int64_t Tq, int64_t Tk, int Hq, int Hkv, int D, int B, int *max_q, int *max_k)
{
    if (!head_dim_ok(D)) return VIT_ERR_BAD_HEAD_DIM;
    if (Tq < 0 || Tq > kMaxRows || Tk < 0 || Tk > kMaxRows || !heads_ok(Hq) || !heads_ok(Hkv) || Hq % Hkv != 0 ||
        B < 0)
        return VIT_ERR_BAD_SHAPE;
    if (B > VIT_MAX_SEGMENTS) return VIT_ERR_TOO_MANY_SEGMENTS;
    if (*max_q < 0 || *max_k < 0) return VIT_ERR_BAD_ARGUMENT;
    if (*max_q == 0 || *max_q > Tq) *max_q = (int)Tq;
    if (*max_k == 0 || *max_k > Tk) *max_k = (int)Tk;
    return VIT_OK;
}

// the checks that the cross-attention calls share (pointers, strides and alignment of q, k, v and the lists)
vit_status_t check_cross(const void *q, const void *k, const void *v, int64_t Tk, int Hq, int Hkv, int D,
                         int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *cu_q,
                         const int32_t *cu_k, const int32_t *k_len, float scale)
{
    if (isnan(scale) || isinf(scale)) return VIT_ERR_BAD_ARGUMENT;
    if (!q || (Tk > 0 && (!k || !v)) || !cu_q || !cu_k) return VIT_ERR_NULL_POINTER;
    if (!stride_ok(q_stride, (int64_t)Hq * D) ||
        (Tk > 0 && (!stride_ok(k_stride, (int64_t)Hkv * D) || !stride_ok(v_stride, (int64_t)Hkv * D))))
        return VIT_ERR_BAD_STRIDE;
    if (!aligned16(q) || (Tk > 0 && (!aligned16(k) || !aligned16(v))) || ((uintptr_t)cu_q & 3u) ||
        ((uintptr_t)cu_k & 3u) || ((uintptr_t)k_len & 3u))
        return VIT_ERR_MISALIGNED;
    return VIT_OK;
}

}  // namespace

size_t vit_cross_attn_workspace_size(int64_t Tq, int64_t Tk, int Hq, int Hkv, int D, int B, int max_q, int max_k)
{
    if (cross_sizes(Tq, Tk, Hq, Hkv, D, B, &max_q, &max_k) != VIT_OK) return 0;
    if (B == 0 || Tq == 0) return 16;
    if (takes_few(B, Hq, Hkv, D, max_q, max_k)) {
        const size_t n = few_plan(B, Hq, Hkv, D, max_q, max_k).partial_bytes;
        return n > 16 ? n : 16;
    }
    const LongPlan p = long_plan(Tq, B, Hq, Hkv, D, max_q, max_k);
    return p.max_items >= ((int64_t)1 << 31) ? 0 : p.bytes;
}

vit_status_t vit_cross_attn(const void *q, const void *k, const void *v, int64_t Tq, int64_t Tk, int Hq, int Hkv,
                            int D, int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *cu_q,
                            const int32_t *cu_k, const int32_t *k_len, int B, int max_q, int max_k, float scale,
                            void *out, int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                            int32_t *status_dev, vit_stream_t stream)
{
    TraceRange trace("vit_cross_attn");
    vit_status_t st = cross_sizes(Tq, Tk, Hq, Hkv, D, B, &max_q, &max_k);
    if (st != VIT_OK) return st;
    if (B == 0 || Tq == 0) return VIT_OK;
    st = check_cross(q, k, v, Tk, Hq, Hkv, D, q_stride, k_stride, v_stride, cu_q, cu_k, k_len, scale);
    if (st != VIT_OK) return st;
    if (!out || !workspace) return VIT_ERR_NULL_POINTER;
    if (!stride_ok(out_stride, (int64_t)Hq * D)) return VIT_ERR_BAD_STRIDE;
    if (!aligned16(out) || ((uintptr_t)lse & 3u) || !aligned16(workspace)) return VIT_ERR_MISALIGNED;
    const size_t need = vit_cross_attn_workspace_size(Tq, Tk, Hq, Hkv, D, B, max_q, max_k);
    if (need == 0) return VIT_ERR_BAD_SHAPE;
    if (workspace_bytes < need) return VIT_ERR_WORKSPACE_TOO_SMALL;
    int sms = 0;
    st = check_device(&sms);
    if (st != VIT_OK) return st;
    CrossArgs a{};
    a.q = q;
    a.k = Tk > 0 ? k : q;                       // no keys anywhere: never read, but a map needs an address
    a.v = Tk > 0 ? v : q;
    a.k_stride = Tk > 0 ? k_stride : q_stride;
    a.v_stride = Tk > 0 ? v_stride : q_stride;
    a.out = out;
    a.lse = lse;
    a.Hq = Hq;
    a.Hk = Hkv;
    a.D = D;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.scale_log2 = (scale <= 0.f ? 1.0f / sqrtf((float)D) : scale) * 1.4426950408889634f;
    a.segs = CrossSegs{cu_q, cu_k, k_len, B, Tq, Tk, max_q, max_k};
    a.workspace = workspace;
    a.status = status_dev;
    cudaStream_t s = (cudaStream_t)stream;
    if (takes_few(B, Hq, Hkv, D, max_q, max_k))
        return from_cuda(launch_cross_few(a, few_plan(B, Hq, Hkv, D, max_q, max_k), s));
    const LongPlan p = long_plan(Tq, B, Hq, Hkv, D, max_q, max_k);
    char *ws = static_cast<char *>(workspace);
    WsHeader *hdr = reinterpret_cast<WsHeader *>(ws);
    CrossItem *items = reinterpret_cast<CrossItem *>(ws + p.off_items);
    CrossTile *tiles = reinterpret_cast<CrossTile *>(ws + p.off_tiles);
    CrossEmpty *empty = reinterpret_cast<CrossEmpty *>(ws + p.off_empty);
    CrossLong cx{};
    cx.group = Hq / Hkv;
    cx.lg_pack = p.lg_pack;
    cx.empty = empty;
    cx.part_s = reinterpret_cast<float *>(ws + p.off_part_s);
    cx.part_o = reinterpret_cast<float *>(ws + p.off_part_o);
    cudaError_t e = launch_cross_schedule(a, p, sms, hdr, items, tiles, empty, s);
    if (e == cudaSuccess) e = launch_cross_long(a, cx, hdr, items, p.max_items, sms, s);
    if (e == cudaSuccess && p.runs > 1) e = launch_cross_tile_join(a, p, cx, hdr, tiles, s);
    return from_cuda(e);
}

size_t vit_cross_attn_bwd_workspace_size(int64_t Tq, int64_t Tk, int Hq, int Hkv, int D, int B, int max_q, int max_k)
{
    if (cross_sizes(Tq, Tk, Hq, Hkv, D, B, &max_q, &max_k) != VIT_OK) return 0;
    const GradPlan p = grad_plan(Tq, Tk, B, Hq, Hkv, D, max_q, max_k);
    return p.max_dq >= ((int64_t)1 << 31) || p.max_dkv >= ((int64_t)1 << 31) ? 0 : p.bytes;
}

vit_status_t vit_cross_attn_bwd(const void *dout, const void *q, const void *k, const void *v, const void *out,
                                const float *lse, int64_t Tq, int64_t Tk, int Hq, int Hkv, int D, int64_t dout_stride,
                                int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t out_stride,
                                const int32_t *cu_q, const int32_t *cu_k, const int32_t *k_len, int B, int max_q,
                                int max_k, float scale, void *dq, void *dk, void *dv, int64_t dq_stride,
                                int64_t dk_stride, int64_t dv_stride, int zero_rest, void *workspace,
                                size_t workspace_bytes, int32_t *status_dev, vit_stream_t stream)
{
    TraceRange trace("vit_cross_attn_bwd");
    vit_status_t st = cross_sizes(Tq, Tk, Hq, Hkv, D, B, &max_q, &max_k);
    if (st != VIT_OK) return st;
    if (B == 0 || (Tq == 0 && Tk == 0)) return VIT_OK;
    // with no rows on one side nothing of it is read: the other side's address stands in for the maps
    if (Tq == 0) {
        q = dout = out = k;
        q_stride = dout_stride = out_stride = (int64_t)Hq * D;
    }
    st = check_cross(q, k, v, Tk, Hq, Hkv, D, q_stride, k_stride, v_stride, cu_q, cu_k, k_len, scale);
    if (st != VIT_OK) return st;
    if (!workspace || (Tq > 0 && (!dout || !out || !lse || !dq)) || (Tk > 0 && (!dk || !dv))) return VIT_ERR_NULL_POINTER;
    const int64_t nq = (int64_t)Hq * D, nk = (int64_t)Hkv * D;
    if (!stride_ok(dout_stride, nq) || !stride_ok(out_stride, nq) || (Tq > 0 && !stride_ok(dq_stride, nq)) ||
        (Tk > 0 && (!stride_ok(dk_stride, nk) || !stride_ok(dv_stride, nk))))
        return VIT_ERR_BAD_STRIDE;
    if (!aligned16(dout) || !aligned16(out) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
        ((uintptr_t)lse & 3u) || !aligned16(workspace))
        return VIT_ERR_MISALIGNED;
    const size_t need = vit_cross_attn_bwd_workspace_size(Tq, Tk, Hq, Hkv, D, B, max_q, max_k);
    if (need == 0) return VIT_ERR_BAD_SHAPE;
    if (workspace_bytes < need) return VIT_ERR_WORKSPACE_TOO_SMALL;
    int sms = 0;
    st = check_device(&sms);
    if (st != VIT_OK) return st;
    CrossGradArgs a{};
    a.f.q = q;
    a.f.k = Tk > 0 ? k : q;
    a.f.v = Tk > 0 ? v : q;
    a.f.k_stride = Tk > 0 ? k_stride : nk;
    a.f.v_stride = Tk > 0 ? v_stride : nk;
    a.f.out = const_cast<void *>(out);
    a.f.lse = const_cast<float *>(lse);
    a.f.Hq = Hq;
    a.f.Hk = Hkv;
    a.f.D = D;
    a.f.q_stride = q_stride;
    a.f.out_stride = out_stride;
    a.f.scale_log2 = (scale <= 0.f ? 1.0f / sqrtf((float)D) : scale) * 1.4426950408889634f;
    a.f.segs = CrossSegs{cu_q, cu_k, k_len, B, Tq, Tk, max_q, max_k};
    a.f.workspace = workspace;
    a.f.status = status_dev;
    a.dout = dout;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dout_stride = dout_stride;
    a.dq_stride = dq_stride;
    a.dk_stride = dk_stride;
    a.dv_stride = dv_stride;
    a.zero_rest = zero_rest != 0;
    return from_cuda(launch_cross_grad(a, grad_plan(Tq, Tk, B, Hq, Hkv, D, max_q, max_k), sms, (cudaStream_t)stream));
}

static vit_status_t check_norm(int64_t T, int C, int res_type, const void *gate, int64_t gate_stride, float scale,
                               float eps)
{
    if (T < 0 || T >= kMaxTokens || C < 8 || C > kMaxWidth || C % 8 != 0) return VIT_ERR_BAD_SHAPE;
    if (res_type != VIT_RES_BF16 && res_type != VIT_RES_FP32) return VIT_ERR_BAD_ARGUMENT;
    if (!isfinite(scale) || !(eps >= 0.f) || !isfinite(eps)) return VIT_ERR_BAD_ARGUMENT;
    if (gate && gate_stride != 0 && !stride_ok(gate_stride, C)) return VIT_ERR_BAD_STRIDE;
    return VIT_OK;
}

vit_status_t vit_norm_residual(const void *x, const void *y, const void *gate, const void *w_post, const void *w_pre,
                               void *h_out, void *z_out, int64_t T, int C, int res_type, int64_t x_stride,
                               int64_t y_stride, int64_t gate_stride, int64_t h_stride, int64_t z_stride, float scale,
                               float eps, vit_stream_t stream)
{
    TraceRange trace("vit_norm_residual");
    vit_status_t st = check_norm(T, C, res_type, gate, gate_stride, scale, eps);
    if (st != VIT_OK) return st;
    if (T == 0) return VIT_OK;
    if (!x || !y || !h_out || (w_pre && !z_out)) return VIT_ERR_NULL_POINTER;
    if (!w_pre && z_out) return VIT_ERR_BAD_ARGUMENT;
    if (!stride_ok(x_stride, C) || !stride_ok(y_stride, C) || !stride_ok(h_stride, C) ||
        (w_pre && !stride_ok(z_stride, C)) || (h_out == x && h_stride != x_stride) ||
        (z_out && z_out == y && z_stride != y_stride))
        return VIT_ERR_BAD_STRIDE;
    if (!aligned16(x) || !aligned16(y) || !aligned16(gate) || !aligned16(w_post) || !aligned16(w_pre) ||
        !aligned16(h_out) || !aligned16(z_out))
        return VIT_ERR_MISALIGNED;
    int sms = 0;
    st = check_device(&sms);
    if (st != VIT_OK) return st;
    NormResidualArgs a{};
    a.x = x;
    a.y = y;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.h_out = h_out;
    a.z_out = z_out;
    a.T = T;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.gate_stride = gate_stride;
    a.h_stride = h_stride;
    a.z_stride = z_stride;
    a.C = C;
    a.res_f32 = res_type == VIT_RES_FP32;
    a.scale = scale;
    a.eps = eps;
    return from_cuda(launch_norm_residual(a, sms, (cudaStream_t)stream));
}

size_t vit_norm_residual_bwd_workspace_size(int C)
{
    if (C < 8 || C > kMaxWidth || C % 8 != 0) return 0;
    return sizeof(float) * 3 * (size_t)C * norm_residual_parts(C);
}

vit_status_t vit_norm_residual_bwd(const void *dz, const void *dh, const void *h, const void *y, const void *gate,
                                   const void *w_post, const void *w_pre, void *dx, void *dy, void *dgate,
                                   float *dw_post, float *dw_pre, int64_t T, int C, int res_type, int64_t dz_stride,
                                   int64_t dh_stride, int64_t h_stride, int64_t y_stride, int64_t gate_stride,
                                   int64_t dx_stride, int64_t dy_stride, int64_t dgate_stride, float scale, float eps,
                                   void *workspace, size_t workspace_bytes, int32_t *status_dev,
                                   vit_stream_t stream)
{
    TraceRange trace("vit_norm_residual_bwd");
    vit_status_t st = check_norm(T, C, res_type, gate, gate_stride, scale, eps);
    if (st != VIT_OK) return st;
    if ((dw_post && !w_post) || (dw_pre && !w_pre) || (dgate && !gate)) return VIT_ERR_BAD_ARGUMENT;
    const bool gate_tok = gate && gate_stride != 0;
    const bool sums = dw_post || dw_pre || (dgate && !gate_tok);
    if (T == 0 && !sums) return VIT_OK;
    if (T > 0) {
        if ((dz != nullptr) != (w_pre != nullptr)) return VIT_ERR_BAD_ARGUMENT;
        if ((!dz && !dh) || (w_pre && !h) || ((w_post || gate) && !y) || !dx || !dy) return VIT_ERR_NULL_POINTER;
        if ((dz && !stride_ok(dz_stride, C)) || (dh && !stride_ok(dh_stride, C)) ||
            (w_pre && !stride_ok(h_stride, C)) || ((w_post || gate) && !stride_ok(y_stride, C)) ||
            !stride_ok(dx_stride, C) || !stride_ok(dy_stride, C) ||
            (gate_tok && dgate && !stride_ok(dgate_stride, C)) || (dx == dh && dx_stride != dh_stride) ||
            (dy == y && (w_post || gate) && dy_stride != y_stride) || (dy == dz && dy_stride != dz_stride))
            return VIT_ERR_BAD_STRIDE;
        if (!aligned16(dz) || !aligned16(dh) || !aligned16(h) || !aligned16(y) || !aligned16(gate) ||
            !aligned16(w_post) || !aligned16(w_pre) || !aligned16(dx) || !aligned16(dy))
            return VIT_ERR_MISALIGNED;
    }
    if (!aligned16(dgate) || ((uintptr_t)dw_post & 3u) || ((uintptr_t)dw_pre & 3u)) return VIT_ERR_MISALIGNED;
    if (sums) {
        if (!workspace) return VIT_ERR_NULL_POINTER;
        if (!aligned16(workspace)) return VIT_ERR_MISALIGNED;
        if (workspace_bytes < vit_norm_residual_bwd_workspace_size(C)) return VIT_ERR_WORKSPACE_TOO_SMALL;
    }
    int sms = 0;
    st = check_device(&sms);
    if (st != VIT_OK) return st;
    NormResidualGrad a{};
    a.dz = dz;
    a.dh = dh;
    a.h = w_pre ? h : nullptr;
    a.y = (w_post || gate) ? y : nullptr;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.dx = dx;
    a.dy = dy;
    a.dgate = dgate;
    a.dw_post = dw_post;
    a.dw_pre = dw_pre;
    a.part = static_cast<float *>(workspace);
    a.T = T;
    a.dz_stride = dz_stride;
    a.dh_stride = dh_stride;
    a.h_stride = h_stride;
    a.y_stride = y_stride;
    a.gate_stride = gate_stride;
    a.dx_stride = dx_stride;
    a.dy_stride = dy_stride;
    a.dgate_stride = dgate_stride;
    a.C = C;
    a.res_f32 = res_type == VIT_RES_FP32;
    a.scale = scale;
    a.eps = eps;
    a.status = status_dev;
    return from_cuda(launch_norm_residual_bwd(a, sms, (cudaStream_t)stream));
}

}  // extern "C"
