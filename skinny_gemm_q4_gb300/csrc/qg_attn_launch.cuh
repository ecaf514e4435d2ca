// Parameters and host-side launchers of the attention-side kernels.
#pragma once
#include <cuda_runtime.h>
#include "qg_kv.cuh"

namespace qg {

struct RopeParams {
    const __half *q, *k, *v;
    __half *qo, *ko;              // ko null: k goes into the cache only
    int64_t qs, qos, ks, kos, vs; // token strides, elements
    const float *qw, *kw;         // null: no norm
    float eps, mscale;
    const int32_t *pos;
    const uint64_t *freq;         // fractions of a turn per position, 2^-64
    const int64_t *slots;
    int nq, nk, nv;               // rows of a token
    int rot;                      // rotated numbers of a head (0: none)
    KvView kv;
};

struct KvReadParams {
    KvView kv;
    const int64_t *slots;
    __half *k, *v;
    int64_t ks, vs;
};

struct AttnParams {
    KvView kv;
    const __half *q;
    __half *out;
    float *lse;
    int64_t qs, os;               // token strides, elements
    const int32_t *q_start, *kv_len, *table;
    int64_t table_stride, N;
    int B, max_q, heads, group;   // q heads, q heads per kv head
    int group_inv;                // 2^16 / group + 1: row * group_inv >> 16 = row / group, row < 64
    int max_len;                  // lengths are cut to this
    float scale;
    int causal, window;
    unsigned int *err;
    // partial results of contexts cut into leaves: [row][head][leaf], token t's row being
    // q_start * row_q + request * row_b + t: its place among the call's tokens (1, 0) or among few_q
    // of each request (0, few_q), whichever are fewer rows
    float *ws_o;                  // sum of p v, D numbers
    float2 *ws_ml;                // (m, sum of p), m in units of log2
    int few_q, few_leaves, row_q, row_b;
    int few_max;                  // most rows of a request that the decode kernel takes in this call
    int row_parts;                // of 16 rows each
    // partial results of keys cut into parts: [token][head][part]
    float *wj_o;
    float2 *wj_ml;
    int splits;                   // parts (1: none)
};

// Most rows (new tokens x heads of a kv head) of the decode kernel: what two parts of 16 hold.  (16
// contexts of up to 4096 tokens, 32 rows each: 45 us there and 62 in the chunk kernel; in Q8
// 50 and 97.)
constexpr int kDecRows = 32;

// Leaves of a context of max_len tokens (qg_attn_decode.cuh).
int attn_leaves(int64_t max_len);

// kind: KV_*; D: 64 or 128; n > 0 tokens.
cudaError_t launch_rope(const RopeParams &p, int kind, int D, bool half, int64_t n, int sms,
                        cudaStream_t s);
cudaError_t launch_kv_read(const KvReadParams &p, int kind, int D, int64_t n, int sms,
                           cudaStream_t s);
// Requests of at most kDecRows rows, and the merge of contexts of several leaves.
cudaError_t launch_attn_decode(const AttnParams &p, int kind, int D, int sms, cudaStream_t s);
cudaError_t launch_attn_decode_f16(const AttnParams &p, int D, int sms, cudaStream_t s);
cudaError_t launch_attn_decode_q8(const AttnParams &p, int D, int sms, cudaStream_t s);
cudaError_t launch_attn_decode_q4(const AttnParams &p, int D, int sms, cudaStream_t s);
// The other requests; pairs: at least the 256-row tile pairs that they have.
cudaError_t launch_attn_chunk(const AttnParams &p, int kind, int D, int64_t pairs, cudaStream_t s);
cudaError_t launch_attn_chunk_f16(const AttnParams &p, int D, int64_t pairs, cudaStream_t s);
cudaError_t launch_attn_chunk_q8(const AttnParams &p, int D, int64_t pairs, cudaStream_t s);
cudaError_t launch_attn_chunk_q4(const AttnParams &p, int D, int64_t pairs, cudaStream_t s);

}  // namespace qg
