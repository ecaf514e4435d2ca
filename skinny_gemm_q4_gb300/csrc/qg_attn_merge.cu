// Joins the partial results of contexts that qg_attn_decode_kernel cut into leaves.  Sixteen
// sums take the leaves in turn (leaf c: sum c mod 16) and are added in a fixed order, so the
// result does not depend on which leaves other rows of the call have.  Reads D + 2 fp32 per leaf,
// mostly from L2, so what counts is the number of loads in flight; two forms, with the same bits:
//   few rows:   a block for 32 numbers of a row, a group of eight lanes for each sum, eight
//               leaves' loads at once (64 rows of 304 leaves: 8.0 us; four at once, after the
//               maximum: 11.8; one block a row: 20)
//   many rows:  a warp for a row, all sixteen sums in its registers, sixteen leaves' loads at once
//               (1024 rows of up to 48 leaves: 9.7 us, in blocks 11.9)
#include "qg_attn_decode.cuh"

namespace qg {

constexpr int kMergeThreads = 128, kMergeGroups = kMergeThreads / 8;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) qg_attn_merge_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float4 part[kMergeThreads / 32][8];
    __shared__ float psum[kMergeThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d4 = 32 * (blockIdx.x % (D / 32)) + 4 * (lane & 7);
    const int row = blockIdx.x / (D / 32), h = row % p.heads;
    const int b = row / p.heads / p.few_q, t = row / p.heads % p.few_q;
    pdl_trigger();
    pdl_wait();
    const Req r = req_of(p, b);
    if (t >= r.T || !few_rows(p, r.T)) return;
    const int c0 = leaf_of(r.lo(p)), c1 = leaf_of(max(r.L, 1) - 1) + 1;
    if (c1 - c0 <= 1) return;  // finished by the decode kernel
    const int64_t at = ((int64_t)(r.q0 * p.row_q + b * p.row_b + t) * p.heads + h) * p.few_leaves;
    const float2 *const mls = p.ws_ml + at;
    // eight leaves' loads at once, the first eight before the maximum is known
    constexpr int U = 8;
    float4 a[U];
    float2 v[U];
    const int first = (c0 & ~(kMergeGroups - 1)) + (int)(threadIdx.x >> 3);
    auto fetch = [&](int cb) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = cb + i * kMergeGroups;
            const bool in = c >= c0 && c < c1;
            v[i] = in ? mls[c] : make_float2(-INFINITY, 0.0f);
            a[i] = in ? *reinterpret_cast<const float4 *>(p.ws_o + (at + c) * D + d4) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    };
    fetch(first);
    float mx = -INFINITY;
#pragma unroll 4
    for (int c = c0 + lane; c < c1; c += 32) mx = fmaxf(mx, mls[c].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    const float m0 = mx == -INFINITY ? 0.0f : mx;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    for (int cb = first; cb < c1; cb += U * kMergeGroups) {
        if (cb != first) fetch(cb);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = cb + i * kMergeGroups;
            if (c < c0 || c >= c1) continue;
            const float f = ex2(v[i].x - m0);
            sum = fmaf(f, v[i].y, sum);
            acc.x = fmaf(f, a[i].x, acc.x), acc.y = fmaf(f, a[i].y, acc.y);
            acc.z = fmaf(f, a[i].z, acc.z), acc.w = fmaf(f, a[i].w, acc.w);
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        acc.x += __shfl_xor_sync(~0u, acc.x, o), acc.y += __shfl_xor_sync(~0u, acc.y, o);
        acc.z += __shfl_xor_sync(~0u, acc.z, o), acc.w += __shfl_xor_sync(~0u, acc.w, o);
    }
    if (lane < 8) part[warp][lane] = acc;
    if (lane == 0) psum[warp] = sum;
    __syncthreads();
    if (threadIdx.x >= 8) return;
    acc = part[0][lane], sum = psum[0];
#pragma unroll
    for (int w = 1; w < kMergeThreads / 32; ++w) {
        const float4 a = part[w][lane];
        sum += psum[w];
        acc.x += a.x, acc.y += a.y, acc.z += a.z, acc.w += a.w;
    }
    store_row_out(p, r.q0 + t, h, D, d4, acc, mx, sum);
}

// Joins the parts of rows whose keys qg_attn_chunk_kernel cut: one warp per (token, head),
// the parts in order.
template <int D>
__global__ void __launch_bounds__(128) qg_attn_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int E = D / 32;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const int64_t n = w / p.heads;
    const int h = (int)(w - n * p.heads);
    if (n >= p.N) return;
    int b = 0, hi = p.B;  // q_start[b] <= n < q_start[b + 1]
    while (hi - b > 1) {
        const int mid = (b + hi) / 2;
        if (p.q_start[mid] <= n) b = mid; else hi = mid;
    }
    const Req r = req_of(p, b);
    if (n < r.q0 || n >= r.q0 + r.T || few_rows(p, r.T)) return;
    const int64_t at = (n * p.heads + h) * p.splits;
    float mx = -INFINITY;
    for (int i = lane; i < p.splits; i += 32) mx = fmaxf(mx, p.wj_ml[at + i].x);
#pragma unroll
    for (int i = 16; i; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, i));
    const float m0 = mx == -INFINITY ? 0.0f : mx;
    float acc[E] = {}, sum = 0.0f;
    for (int i0 = 0; i0 < p.splits; i0 += 8) {  // eight parts' loads at once
        float a[8][E];
        float2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = i0 + i < p.splits;
            v[i] = in ? p.wj_ml[at + i0 + i] : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int e = 0; e < E; ++e) a[i][e] = in ? p.wj_o[(at + i0 + i) * D + E * lane + e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = ex2(v[i].x - m0);
            sum = fmaf(f, v[i].y, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(f, a[i][e], acc[e]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    __half *o = p.out + n * p.os + (int64_t)h * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(o + e) = pack_h2(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[n * p.heads + h] = lse_of(mx, sum);
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads) qg_attn_merge_rows_kernel(const __grid_constant__ AttnParams p,
                                                                           int64_t rows)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (row >= rows) return;
    const int h = (int)(row % p.heads), b = (int)(row / p.heads / p.few_q), t = (int)(row / p.heads % p.few_q);
    const Req r = req_of(p, b);
    if (t >= r.T || !few_rows(p, r.T)) return;
    const int c0 = leaf_of(r.lo(p)), c1 = leaf_of(max(r.L, 1) - 1) + 1;
    if (c1 - c0 <= 1) return;
    const int64_t at = ((int64_t)(r.q0 * p.row_q + b * p.row_b + t) * p.heads + h) * p.few_leaves;
    const float2 *const mls = p.ws_ml + at;
    float mx = -INFINITY;
    for (int c = c0 + lane; c < c1; c += 32) mx = fmaxf(mx, mls[c].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    const float m0 = mx == -INFINITY ? 0.0f : mx;
    float acc[16][E], sum[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        sum[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] = 0.0f;
    }
    for (int cb = c0 & ~15; cb < c1; cb += 16) {
        float a[16][E];
        float2 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const bool in = cb + i >= c0 && cb + i < c1;
            v[i] = in ? mls[cb + i] : make_float2(-INFINITY, 0.0f);
            const float *s = p.ws_o + (at + cb + i) * D + E * lane;
#pragma unroll
            for (int e = 0; e < E; ++e) a[i][e] = in ? s[e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (cb + i < c0 || cb + i >= c1) continue;
            const float f = ex2(v[i].x - m0);
            sum[i] = fmaf(f, v[i].y, sum[i]);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] = fmaf(f, a[i][e], acc[i][e]);
        }
    }
    // as the blocks do: sums 4 w .. 4 w + 3 in pairs, then w = 0, 1, 2, 3
    auto tree = [](auto at_) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float q = (at_(4 * w) + at_(4 * w + 1)) + (at_(4 * w + 2) + at_(4 * w + 3));
            s = w ? s + q : q;
        }
        return s;
    };
    const float total = tree([&](int i) { return sum[i]; });
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const int64_t n = r.q0 + t;
    __half *o = p.out + n * p.os + (int64_t)h * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(o + e) =
            pack_h2(tree([&](int i) { return acc[i][e]; }) * inv, tree([&](int i) { return acc[i][e + 1]; }) * inv);
    if (p.lse && lane == 0) p.lse[n * p.heads + h] = lse_of(mx, total);
}

int attn_leaves(int64_t max_len) { return leaf_of((int)(max_len > 1 ? max_len - 1 : 0)) + 1; }

cudaError_t launch_attn_decode(const AttnParams &p, int kind, int D, int sms, cudaStream_t s)
{
    cudaError_t e = kind == KV_F16  ? launch_attn_decode_f16(p, D, sms, s)
                    : kind == KV_Q8 ? launch_attn_decode_q8(p, D, sms, s)
                                    : launch_attn_decode_q4(p, D, sms, s);
    if (e != cudaSuccess || attn_leaves(p.max_len) <= 1) return e;
    cudaLaunchConfig_t cfg = {};
    // rows that fill the GPU's schedulers with a warp each take the second form
    const int64_t rows = (int64_t)p.B * p.few_q * p.heads;
    const bool many = rows >= 4 * sms;
    cfg.gridDim = dim3((unsigned)(many ? (rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32) : rows * (D / 32)));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (many)
        return D == 128 ? cudaLaunchKernelEx(&cfg, qg_attn_merge_rows_kernel<128>, p, rows)
                        : cudaLaunchKernelEx(&cfg, qg_attn_merge_rows_kernel<64>, p, rows);
    return D == 128 ? cudaLaunchKernelEx(&cfg, qg_attn_merge_kernel<128>, p)
                    : cudaLaunchKernelEx(&cfg, qg_attn_merge_kernel<64>, p);
}

cudaError_t launch_attn_chunk(const AttnParams &p, int kind, int D, int64_t pairs, cudaStream_t s)
{
    cudaError_t e = kind == KV_F16  ? launch_attn_chunk_f16(p, D, pairs, s)
                    : kind == KV_Q8 ? launch_attn_chunk_q8(p, D, pairs, s)
                                    : launch_attn_chunk_q4(p, D, pairs, s);
    if (e != cudaSuccess || p.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N * p.heads + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 128 ? cudaLaunchKernelEx(&cfg, qg_attn_join_kernel<128>, p)
                    : cudaLaunchKernelEx(&cfg, qg_attn_join_kernel<64>, p);
}

}  // namespace qg
