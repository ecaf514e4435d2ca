// Norm + rotation of q and k, and the paged cache's writes and reads.
//
// All of it moves heads of D fp16 numbers with a few flops each, so the floor is HBM's: 8192 tokens of
// 40 heads, 168 MB, 33.8 us, 4.97 TB/s, where issue slots are 63 % and DRAM 46 % busy and a warp's
// turn is a chain of loads, shuffles and products.  Quantised it is bound by its instructions: 8191
// tokens of 2 x 8 heads written in 20.5 (Q8), 21.4 us (Q4) and read in 16.1, 13.8 (issue slots
// 62-67 % busy); in fp16 14.6 and 12.4 (floor 10.0).  Single tokens: a launch (2.7 us).
// A block takes one token: D / 8 lanes hold a head (8 numbers, one 16-byte
// access each), so a head's sum of squares, its rotation partners and its
// quantisation maxima are shuffles inside 16 (D = 128) or 8 lanes, and a head
// is read and written once.  The token's cos and sin are computed once per
// block, one pair per thread.
#include <algorithm>

#include "qg_attn_launch.cuh"
#include "qg_ptx.cuh"

namespace qg {

namespace {

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void load8(const float *w, float (&x)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w)), b = __ldg(reinterpret_cast<const float4 *>(w + 4));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Maxima that keep a NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Quantise and store one head's row (numbers 8 l .. 8 l + 7 in lane l of its D /
// 8 lanes) as row `t` of a record; `live` is false for lanes whose row is not
// stored (they take part in the shuffles).  A row with a NaN or an infinity gets a step of NaN and
// multipliers of 0: every number of it stands for NaN.
template <int KIND, int D>
__device__ __forceinline__ void store_row(const float (&x)[8], int l, uint8_t *rec, int t, int which,
                                          bool live)
{
    if constexpr (KIND == KV_F16) {
        if (live)
            *reinterpret_cast<uint4 *>(rec + kv_rows_at(KIND, D, which) +
                                       kv_unit(KIND, D, (uint32_t)t, (uint32_t)l)) = pack8(x);
        return;
    }
    constexpr float kTop = KIND == KV_Q8 ? 127.0f : 8.0f, kMost = KIND == KV_Q8 ? 15.0f : 127.0f;
    float big = 0.0f;
    bool flip = false;  // Q4: the block's first number of largest magnitude is positive
    if constexpr (KIND == KV_Q8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max_nan(big, fabsf(x[i]));
        big = max_nan(big, __shfl_xor_sync(~0u, big, 1));
        big = max_nan(big, __shfl_xor_sync(~0u, big, 2));
    } else {
        float up = 0.0f, down = 0.0f;  // largest positive, and negated negative, number
#pragma unroll
        for (int i = 0; i < 8; ++i) up = max_nan(up, x[i]), down = max_nan(down, -x[i]);
        up = max_nan(up, __shfl_xor_sync(~0u, up, 1)), down = max_nan(down, __shfl_xor_sync(~0u, down, 1));
        up = max_nan(up, __shfl_xor_sync(~0u, up, 2)), down = max_nan(down, __shfl_xor_sync(~0u, down, 2));
        big = max_nan(up, down);
        flip = up > down;
        if (__any_sync(~0u, up == down)) {  // which comes first?
            bool has = false, pos = false;
#pragma unroll
            for (int i = 7; i >= 0; --i)
                if (fabsf(x[i]) == big) has = true, pos = x[i] > 0.0f;
            const int lane = threadIdx.x & 31;
            const uint32_t in = __ballot_sync(~0u, has) >> (lane & 28) & 15u;
            const uint32_t plus = __ballot_sync(~0u, pos) >> (lane & 28) & 15u;
            if (up == down) flip = (in & (0u - in) & plus) != 0;
        }
    }
    float top = big;
#pragma unroll
    for (int o = 4; o < D / 8; o <<= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
    float d = __fdiv_rn(top, kTop * kMost);
    d += d - d;  // an infinity: NaN
    float m = d > 0.0f ? fminf(ceilf(__fdiv_rn(big, __fmul_rn(kTop, d))), kMost) : 0.0f;
    if (flip) m = -m;
    const float f = __fmul_rn(d, m);
    // The code is the rounded quotient x / f.  By the reciprocal it is off by at most 3 2^-24 of
    // itself, so only quotients within 1e-4 of a half can round elsewhere: where a lane has one, it
    // divides.  (Added to 1.5 2^23, and 8 for Q4, a number rounds to the integer that its low bits
    // then hold.)
    constexpr float kInt = 12582912.0f + (KIND == KV_Q4 ? 8.0f : 0.0f);
    const float inv = m != 0.0f ? __frcp_rn(f) : 0.0f;
    float r[8], off = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r[i] = fmaf(x[i], inv, kInt);
        off = fmaxf(off, fabsf(fmaf(x[i], inv, kInt - r[i])));
    }
    if (off > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(fmaf(x[i], inv, kInt - r[i])) > 0.4999f) r[i] = __fdiv_rn(x[i], f) + kInt;
    }
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = __float_as_uint(KIND == KV_Q4 ? fminf(r[i], kInt + 7.0f) : r[i]);
    uint8_t *rows = rec + kv_rows_at(KIND, D, which);
    const uint32_t lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    const uint32_t hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
    if constexpr (KIND == KV_Q8) {
        if (live)
            *reinterpret_cast<uint2 *>(rows + kv_unit(KIND, D, (uint32_t)t, (uint32_t)l >> 1) +
                                       8 * (l & 1)) = make_uint2(lo, hi);
    } else {
        // numbers i and i + 16 of a block share a byte: lane 4 b + j takes the
        // codes of lane 4 b + j + 2
        const uint32_t lo2 = __shfl_xor_sync(~0u, lo, 2), hi2 = __shfl_xor_sync(~0u, hi, 2);
        if (live && !(l & 2))
            *reinterpret_cast<uint2 *>(rows + kv_unit(KIND, D, (uint32_t)t, (uint32_t)l >> 2) +
                                       8 * (l & 1)) = make_uint2(lo | lo2 << 4, hi | hi2 << 4);
    }
    if (live && (l & 3) == 0)
        *reinterpret_cast<int8_t *>(rec + kv_mults_at(KIND, D, which) + t * (D / 32) + (l >> 2)) =
            (int8_t)m;
    if (live && l == 0)
        *reinterpret_cast<float *>(rec + kv_steps_at(KIND, D, which) + 4 * t) = d;
}

// step * f (f a whole number below 2048) as an fp32 number that rounds to fp16 as the exact
// product does: rounded towards zero with the last bit set where it is not
// exact (the product has 35 bits; fp32's 24 round first and fp16's 11 second
// would differ near ties).
__device__ __forceinline__ float step_times(float step, float f)
{
    const float p = __fmul_rz(step, f);
    const uint32_t inexact = __fmaf_rn(step, f, -p) != 0.0f;
    return __uint_as_float(__float_as_uint(p) | inexact);
}

// The stored form of numbers 8 l .. 8 l + 7 of row t, and the numbers.
struct RawRow {
    uint4 w;  // fp16: the numbers; codes: x, y
    float d;
    int m;
};
template <int KIND, int D>
__device__ __forceinline__ RawRow load_row(const uint8_t *rec, int l, int t, int which)
{
    RawRow r = {};
    const uint8_t *rows = rec + kv_rows_at(KIND, D, which);
    if constexpr (KIND == KV_F16) {
        r.w = *reinterpret_cast<const uint4 *>(rows + kv_unit(KIND, D, (uint32_t)t, (uint32_t)l));
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(
            rows + kv_unit(KIND, D, (uint32_t)t, (uint32_t)l >> (KIND == KV_Q8 ? 1 : 2)) + 8 * (l & 1));
        r.w = make_uint4(w.x, w.y, 0, 0);
        r.d = *reinterpret_cast<const float *>(rec + kv_steps_at(KIND, D, which) + 4 * t);
        r.m = *reinterpret_cast<const int8_t *>(rec + kv_mults_at(KIND, D, which) + t * (D / 32) + (l >> 2));
    }
    return r;
}
template <int KIND>
__device__ __forceinline__ uint4 row_numbers(const RawRow &r, int l)
{
    if constexpr (KIND == KV_F16) return r.w;
    // multiplier * code: 2^23 + a whole number as bits, less 2^23 + the code's zero, times the multiplier
    float x[8];
    const int sh = (l & 2) ? 4 : 0;
    const float m = (float)r.m, zero = KIND == KV_Q8 ? 8388736.0f : 8388616.0f;
    const uint32_t w[2] = {KIND == KV_Q8 ? r.w.x ^ 0x80808080u : r.w.x >> sh & 0x0f0f0f0fu,
                           KIND == KV_Q8 ? r.w.y ^ 0x80808080u : r.w.y >> sh & 0x0f0f0f0fu};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = step_times(r.d, (__uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7540 | (i & 3))) - zero) * m);
    return pack8(x);
}

}  // namespace

constexpr int kReadAhead = 4;

// One warp's turns [a, b) on the heads of a kind, 32 / (D / 8) heads a turn, two turns' loads ahead.
// `work(x, raw, h)` gets a lane's 8 numbers of head h (zeros past the last head).
template <int D, class Work>
__device__ __forceinline__ void turns(const __half *src, int a, int b, int heads, int lane, Work work)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    int h = a * RPW + lane / LPR;
    const __half *at = src + (int64_t)h * D + 8 * (lane % LPR);
    auto load = [&](bool in) { return in ? *reinterpret_cast<const uint4 *>(at) : make_uint4(0, 0, 0, 0); };
    uint4 next = load(a < b && h < heads);
    at += RPW * D;
    uint4 next2 = load(a + 1 < b && h + RPW < heads);
    for (; a < b; ++a, h += RPW) {
        const uint4 raw = next;
        next = next2;
        at += RPW * D;
        next2 = load(a + 2 < b && h + 2 * RPW < heads);
        float x[8];
        unpack8(raw, x);
        work(x, raw, h);
    }
}

// Norm and rotation are one product and one multiply-add a number,
//     y = rs (x cw + x' sw),   x' the other number of the pair, cw = cos w, sw = -+ sin w',
// with cw and sw made once per warp and kind, and x' fetched as it was read (two fp16 numbers a
// shuffle).  Bound by instruction issue below the HBM rate: about 100 for 8 numbers a lane.
template <int D, int KIND, bool HALF>
__global__ void __launch_bounds__(512) qg_rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ __align__(16) float2 cs[D / 2];
    const int64_t n = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int l = lane % LPR;
    // the token's turns, q heads, k heads, v heads, in equal runs to the warps
    const int tq = (p.nq + RPW - 1) / RPW, tk = (p.nk + RPW - 1) / RPW, tv = (p.nv + RPW - 1) / RPW;
    const int per = (tq + tk + tv + warps - 1) / warps, first = warp * per, last = first + per;
    pdl_trigger();
    pdl_wait();
    int64_t slot = -1;
    uint8_t *rec = nullptr;  // the token's record of head 0, and the heads' distance
    int64_t rec_step = 0;
    if constexpr (KIND != KV_NONE) {
        slot = p.slots[n];
        if (slot >= p.kv.slots) {
            if (threadIdx.x == 0) atomicOr(p.kv.err, kStatusRange);
            slot = -1;
        }
        if (slot >= 0) rec = kv_record<KIND, D>(p.kv, slot, 0);
        rec_step = (int64_t)kv_record_bytes(KIND, D) << (p.kv.page_shift - 4);
    }
    if (p.rot) {
        // the position's angle as a fraction of a turn, modulo 1 by the wrap of 64 bits
        const int64_t pos = p.pos[n];
        for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) {
            const uint64_t ph = (uint64_t)pos * p.freq[i];
            float sn, cn;
            sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &sn, &cn);
            cs[i] = make_float2(cn * p.mscale, sn * p.mscale);
        }
        __syncthreads();
    }
    const int hl = p.rot / 16;  // lanes of half the rotated part
    // HALF: the lane of the row with the other numbers of this one's pairs
    const int mate = l < hl ? l + hl : l < 2 * hl ? l - hl : l;
    const int from = lane - l + mate;

    auto rotated = [&](const __half *src, int off, int count, int heads, const float *w, auto out) {
        const int a = max(first - off, 0), b = min(last - off, count);
        if (a >= b) return;
        float cw[8], sw[8];
        {
            float own[8], other[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) own[i] = other[i] = 1.0f;
            if (w) {
                load8(w + 8 * l, own);
                if constexpr (HALF) {
                    load8(w + 8 * mate, other);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) other[i] = own[i ^ 1];
                }
            }
            // HALF: number 8 l + i is in pair (8 l + i) mod (rot / 2); else pair 4 l + i / 2
            const bool turn = 8 * l < p.rot;
            const float4 *c4 = reinterpret_cast<const float4 *>(cs) + (HALF ? 4 * min(l, mate) : 2 * l);
            float2 v[8];
#pragma unroll
            for (int i = 0; i < (HALF ? 4 : 2); ++i) {
                const float4 f = turn ? c4[i] : make_float4(1.0f, 0.0f, 1.0f, 0.0f);
                v[2 * i] = make_float2(f.x, f.y), v[2 * i + 1] = make_float2(f.z, f.w);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = v[HALF ? i : i / 2];
                cw[i] = f.x * own[i];
                sw[i] = ((HALF ? l < hl : !(i & 1)) ? -f.y : f.y) * other[i];
            }
        }
        turns<D>(src, a, b, heads, lane, [&](float (&x)[8], const uint4 &raw, int h) {
            float rs = 1.0f;
            if (w) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
                rs = rsqrtf(ss * (1.0f / D) + p.eps);
            }
            float y[8];
            if constexpr (HALF) {
                unpack8(make_uint4(__shfl_sync(~0u, raw.x, from), __shfl_sync(~0u, raw.y, from),
                                   __shfl_sync(~0u, raw.z, from), __shfl_sync(~0u, raw.w, from)),
                        y);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
            }
            if (p.rot < D && 8 * l >= p.rot) {  // (an infinity times sw = 0 is NaN)
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = rs * fmaf(x[i], cw[i], y[i] * sw[i]);
            out(x, h);
        });
    };
    rotated(p.q + n * p.qs, 0, tq, p.nq, p.qw, [&](float (&x)[8], int h) {
        if (h < p.nq) *reinterpret_cast<uint4 *>(p.qo + n * p.qos + (int64_t)h * D + 8 * l) = pack8(x);
    });
    auto k_out = [&](float (&x)[8], int h) {
        if (p.ko && h < p.nk) *reinterpret_cast<uint4 *>(p.ko + n * p.kos + (int64_t)h * D + 8 * l) = pack8(x);
        if constexpr (KIND != KV_NONE)
            store_row<KIND, D>(x, l, rec + h * rec_step, (int)(slot & 15), 0, slot >= 0 && h < p.nk);
    };
    if (KIND == KV_NONE || p.rot)
        rotated(p.k + n * p.ks, tq, tk, p.nk, p.kw, k_out);
    else  // keys into the cache as they are
        turns<D>(p.k + n * p.ks, max(first - tq, 0), min(last - tq, tk), p.nk, lane,
                 [&](float (&x)[8], const uint4 &, int h) { k_out(x, h); });
    if constexpr (KIND != KV_NONE)
        turns<D>(p.v + n * p.vs, max(first - tq - tk, 0), min(last - tq - tk, tv), p.nv, lane, [&](float (&x)[8], const uint4 &, int h) {
            store_row<KIND, D>(x, l, rec + h * rec_step, (int)(slot & 15), 1, slot >= 0 && h < p.nv);
        });
}

// K and V rows of the slots' tokens, as fp16.
template <int D, int KIND>
__global__ void __launch_bounds__(512) qg_kv_read_kernel(const __grid_constant__ KvReadParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int64_t n = blockIdx.x;
    const int lane = threadIdx.x & 31, l = lane % LPR;
    const int step = (int)(blockDim.x >> 5) * RPW;
    pdl_trigger();
    pdl_wait();
    int64_t slot = p.slots[n];
    if (slot >= p.kv.slots) {
        if (threadIdx.x == 0) atomicOr(p.kv.err, kStatusRange);
        slot = -1;
    }
    const int rows = 2 * p.kv.heads;
    for (int r = (int)(threadIdx.x >> 5) * RPW + lane / LPR; r < rows; r += kReadAhead * step) {
        RawRow raw[kReadAhead];
#pragma unroll
        for (int i = 0; i < kReadAhead; ++i) {
            const int q = r + i * step, which = q >= p.kv.heads;
            raw[i] = {};
            if (slot >= 0 && q < rows)
                raw[i] = load_row<KIND, D>(kv_record<KIND, D>(p.kv, slot, q - which * p.kv.heads), l,
                                           (int)(slot & 15), which);
        }
#pragma unroll
        for (int i = 0; i < kReadAhead; ++i) {
            const int q = r + i * step, which = q >= p.kv.heads;
            if (q >= rows) break;
            __half *dst = which ? p.v + n * p.vs : p.k + n * p.ks;
            *reinterpret_cast<uint4 *>(dst + (int64_t)(q - which * p.kv.heads) * D + 8 * l) =
                row_numbers<KIND>(raw[i], l);
        }
    }
}

namespace {

// A block per token.  Warps: what gives the GPU about 32 an SM, between a turn each and `most` turns
// each.  Rotation: up to 20, so that cos, sin and the weights serve many heads while a token of very
// many still has warps enough.  8192 tokens, most 5 / 10 / 20 / 40, us: 32 + 8 heads of 128 (20
// turns) 40.0 / 34.9 / 33.9 / 33.9, 64 + 8 73 / 58 / 55 / 55, 96 + 8 125 / 85 / 77 / 76, 16 + 2 21.3
// / 20.0 / 19.9 / 19.9, 12 + 12 of 64 the same in all.  Reading: the loads that a lane has in flight.
template <class P, class K>
cudaError_t launch_tokens(K kernel, const P &p, int64_t n, int turns, int most, int sms, cudaStream_t stream)
{
    const int64_t fill = (32 * (int64_t)sms + n - 1) / n, least = (turns + most - 1) / most;
    const int warps = (int)std::min((int64_t)turns, std::max(least, fill));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n);
    cfg.blockDim = dim3(32 * (unsigned)(warps > 16 ? 16 : warps));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, bool HALF>
cudaError_t rope_kind(const RopeParams &p, int kind, int64_t n, int turns, int sms, cudaStream_t s)
{
    switch (kind) {
    case KV_F16: return launch_tokens(qg_rope_kernel<D, KV_F16, HALF>, p, n, turns, 20, sms, s);
    case KV_Q8: return launch_tokens(qg_rope_kernel<D, KV_Q8, HALF>, p, n, turns, 20, sms, s);
    case KV_Q4: return launch_tokens(qg_rope_kernel<D, KV_Q4, HALF>, p, n, turns, 20, sms, s);
    default: return launch_tokens(qg_rope_kernel<D, KV_NONE, HALF>, p, n, turns, 20, sms, s);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int kind, int D, bool half, int64_t n, int sms,
                        cudaStream_t s)
{
    const int rpw = 256 / D;
    const int turns = (p.nq + rpw - 1) / rpw + (p.nk + rpw - 1) / rpw + (p.nv + rpw - 1) / rpw;
    if (D == 128)
        return half ? rope_kind<128, true>(p, kind, n, turns, sms, s)
                    : rope_kind<128, false>(p, kind, n, turns, sms, s);
    return half ? rope_kind<64, true>(p, kind, n, turns, sms, s)
                : rope_kind<64, false>(p, kind, n, turns, sms, s);
}

cudaError_t launch_kv_read(const KvReadParams &p, int kind, int D, int64_t n, int sms,
                           cudaStream_t s)
{
    const int rpw = 256 / D, turns = (2 * p.kv.heads + rpw - 1) / rpw;
    if (D == 128) {
        if (kind == KV_F16) return launch_tokens(qg_kv_read_kernel<128, KV_F16>, p, n, turns, kReadAhead, sms, s);
        if (kind == KV_Q8) return launch_tokens(qg_kv_read_kernel<128, KV_Q8>, p, n, turns, kReadAhead, sms, s);
        return launch_tokens(qg_kv_read_kernel<128, KV_Q4>, p, n, turns, kReadAhead, sms, s);
    }
    if (kind == KV_F16) return launch_tokens(qg_kv_read_kernel<64, KV_F16>, p, n, turns, kReadAhead, sms, s);
    if (kind == KV_Q8) return launch_tokens(qg_kv_read_kernel<64, KV_Q8>, p, n, turns, kReadAhead, sms, s);
    return launch_tokens(qg_kv_read_kernel<64, KV_Q4>, p, n, turns, kReadAhead, sms, s);
}

}  // namespace qg
