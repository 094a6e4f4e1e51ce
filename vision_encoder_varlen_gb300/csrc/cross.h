// Declarations shared by the cross-attention translation units.
#pragma once

#include "internal.h"

namespace vit {

// The packed sequences of a cross-attention call: sequence b has the query rows [cu_q[b], cu_q[b+1])
// and the key rows [cu_k[b], cu_k[b] + len), len = k_len[b] where given, else cu_k[b+1] - cu_k[b].
struct CrossSegs {
    const int32_t *cu_q, *cu_k, *k_len;   // k_len may be NULL
    int B;
    int64_t Tq, Tk;
    int max_q, max_k;
};
struct CrossSeg {
    int q0, qn, k0, kn;
};

// Reads sequence b and checks it: false (and the status code reported by one caller per sequence,
// `report`) when an offset decreases or leaves the tensors, a key count does not fit its rows, or a
// length exceeds its bound. Such a sequence is left alone by every kernel.
__device__ __forceinline__ bool load_seg(const CrossSegs &s, int b, CrossSeg &x, int32_t *status, bool report)
{
    const int64_t q0 = s.cu_q[b], q1 = s.cu_q[b + 1], k0 = s.cu_k[b], k1 = s.cu_k[b + 1];
    const int64_t kn = s.k_len ? (int64_t)s.k_len[b] : k1 - k0;
    x.q0 = (int)q0;
    x.qn = (int)(q1 - q0);
    x.k0 = (int)k0;
    x.kn = (int)kn;
    int err = 0;
    if (q0 < 0 || q1 < q0 || q1 > s.Tq || k0 < 0 || k1 < k0 || k1 > s.Tk || kn < 0 || kn > k1 - k0)
        err = VIT_ERR_BAD_SEQLENS;
    else if (q1 - q0 > s.max_q || kn > s.max_k)
        err = VIT_ERR_SEQLEN_EXCEEDS_MAX;
    if (err && report) report_error(status, err);
    return err == 0;
}

// runs of `chunk` keys that n keys make (the sum may pass 31 bits)
__host__ __device__ inline int key_runs(int n, int chunk) {
    return (int)(((unsigned)n + (unsigned)chunk - 1u) / (unsigned)chunk);
}

struct CrossArgs {
    const void *q, *k, *v;        // bf16 [Tq, Hq, D], [Tk, Hk, D], [Tk, Hk, D]
    void *out;                    // bf16 [Tq, Hq, D]
    float *lse;                   // fp32 [Tq, Hq] or NULL
    int Hq, Hk, D;
    int64_t q_stride, k_stride, v_stride, out_stride;
    float scale_log2;             // scale * log2(e)
    CrossSegs segs;
    void *workspace;
    int32_t *status;
};

// How a call with few query rows per sequence and key head is cut (a function of the sizes alone, so
// that the workspace size is one too).
struct FewPlan {
    int rows;                     // max_q * group: query rows that share one key head
    int row_tiles;                // 16-row tiles of a block: 1 or 2
    int chunk;                    // keys per split
    int n_split;                  // splits of the longest sequence
    int room;                     // splits that the workspace has room for
    size_t partial_bytes;         // workspace of the partial results (0 with one split)
};
bool takes_few(int B, int Hq, int Hk, int D, int max_q, int max_k);   // else the tcgen05 kernel takes the call
FewPlan few_plan(int B, int Hq, int Hk, int D, int max_q, int max_k);
cudaError_t launch_cross_few(const CrossArgs &a, const FewPlan &p, cudaStream_t stream);

// Work item of the tcgen05 kernel in cross attention: the keys [k0, k0 + kn) for 128 (split) or 256
// query rows. A 128-row tile is 128 / P tokens, from token q0 on, of the P heads from `head` on (P
// divides the heads that share a key head); tokens at or past q1 do not exist.
struct CrossItem {
    int k0, kn, q0, q1;
    int head;
    int split;                    // one tile, whose key tiles alternate between the kernel's two halves
    int slot;                     // place of the partial result of this key run, or -1: the result itself
    int pad;
};
static_assert(sizeof(CrossItem) == 32, "two 16-byte words");
__device__ __forceinline__ int item_head(const CrossItem &x) { return x.head; }
__device__ __forceinline__ bool item_split(const CrossItem &x) { return x.split != 0; }

// A 128-row tile whose keys were cut into several runs: the join adds the slots [slot, slot + runs).
struct CrossTile {
    int q0, q1, head, slot;
    int runs, pad[3];
};

// The query rows of a sequence without keys, which has no items.
struct CrossEmpty {
    int q0, qn;
};

// What the tcgen05 kernel needs besides the self-attention kernels' parameters.
struct CrossLong {
    int group, lg_pack;           // query heads per key head; log2 of P
    const CrossEmpty *empty;      // hdr->n_empty of them
    float *part_o, *part_s;       // [slots][128][D], [slots][128] (log2 of the run's sum)
};

// How such a call is cut (a function of the sizes alone).
struct LongPlan {
    int lg_pack;
    int chunk;                    // keys per run (0: keys are not cut)
    int64_t max_items, max_tiles; // bounds of the item list and of the tiles with several runs
    int runs;                     // runs of the longest sequence
    size_t off_items, off_tiles, off_empty, off_part_s, off_part_o, bytes;   // workspace layout
};
LongPlan long_plan(int64_t Tq, int B, int Hq, int Hk, int D, int max_q, int max_k);
int cross_pack(int group);     // log2 of P
int attn_long_bn(int D);
cudaError_t launch_cross_schedule(const CrossArgs &a, const LongPlan &p, int num_sms, WsHeader *hdr, CrossItem *items,
                                  CrossTile *tiles, CrossEmpty *empty, cudaStream_t stream);
cudaError_t launch_cross_long(const CrossArgs &a, const CrossLong &cx, const WsHeader *hdr, const CrossItem *items,
                              int64_t max_items, int num_sms, cudaStream_t stream);
cudaError_t launch_cross_tile_join(const CrossArgs &a, const LongPlan &p, const CrossLong &cx, const WsHeader *hdr,
                                   const CrossTile *tiles, cudaStream_t stream);

// ---- gradient

// Work item of a gradient pass. dk, dv: the 128 keys from r0 on (below r1) of key head `head`, over
// the queries [l0, l0 + ln) of all its heads; dq: the 128 / P tokens from r0 on of P heads, over the
// keys [l0, l0 + ln), which are `tiles` steps of the loop (0: nothing to add up).
struct GradItem {
    int r0, r1, l0, ln;
    int head, tiles;
    int exact;                    // delta from the scores (few keys), else from the stored out
    int pad;
};
static_assert(sizeof(GradItem) == 32, "two 16-byte words");

struct GradPlan {
    int lg_pack;
    int64_t max_dq, max_dkv;      // bounds of the two item lists
    size_t off_dq, off_dkv, off_stats, bytes;   // workspace layout; at 0: the two lists' lengths
};
struct CrossGradArgs {
    CrossArgs f;                  // the forward call: its inputs, out and lse (read), workspace of this call
    const void *dout;             // bf16 [Tq, Hq, D]
    void *dq, *dk, *dv;
    int64_t dout_stride, dq_stride, dk_stride, dv_stride;
    bool zero_rest;               // rows of no sequence get 0
};
GradPlan grad_plan(int64_t Tq, int64_t Tk, int B, int Hq, int Hk, int D, int max_q, int max_k);
cudaError_t launch_cross_grad(const CrossGradArgs &a, const GradPlan &p, int num_sms, cudaStream_t stream);

}  // namespace vit
