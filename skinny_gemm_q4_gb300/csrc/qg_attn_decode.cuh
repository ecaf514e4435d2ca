// Attention of few rows (decode and verify): requests whose new tokens times
// the q heads of a kv head are at most 32 rows.
//
// The bound is HBM: every record of the context (16 tokens of one kv head) is
// read once and meets at most 32 rows, 2-8 flop per byte.  Every warp is a
// stream of its own: it walks the list of leaves (a leaf is a short piece of one
// (request, kv head) context), keeps a ring of records filled by bulk copies (one
// copy a record: 8 KB fp16, 4.25 KB Q8, 2.25 KB Q4 at D = 128), and holds the running
// maximum, sum and output of the leaf's rows in registers.  Nothing waits for another
// warp.  Measured, with the merge: 32 contexts of up to 8192 tokens in Q8 (215 MB) 58 us, 3.7 TB/s;
// two of 131072 in Q4 (302 MB) 96 us, 3.1 TB/s: issue slots 61-63 % busy, about 590 and 472
// instructions a record (a third of them the codes' decoding, then products, sums and masks, the
// walk, the copies and the leaves' ends), DRAM 43-56 %.  (With the eight warps of a CTA sharing a chunk and merging it through shared
// memory, 32 contexts of up to 8192 in Q8 took 103 us: a third of the time was spent
// at the chunks' ends.)
//
// Products by mma.sync m16n8k16 with the tokens as the 16 rows: S^T = K Q^T
// (8 query rows in the n dimension) and O^T = V^T P^T, so a decode step of up
// to 8 rows wastes no tensor work on padding to 16.  K fragments come from
// shared memory as they lie (ldmatrix, or code bytes decoded in registers);
// S^T turns into the B operand P^T by one 8 x 8 transposition (movmatrix).
// K's codes are the fp16 operand, exact; a block's multiplier and the token's step join its
// fp32 sums.  V's operand is multiplier * code, exact (Q4: scaled by 2^-16); its step
// multiplies the weights.
//
// With quantised V the weight that meets the tensor core is p * step, so the
// running maximum m is that of score + log2(step): weights are at most 2^kLazy
// whatever the steps' size; the sum of p uses the same m.
//
// Leaves: a context is cut at absolute positions (64 tokens each up to 1024, 128 up to
// 2048, 256 up to 16384, then 512), so a row's bits depend on its own keys alone.  Small
// leaves spread a short context over the SMs and level the warps; larger ones keep the partial
// results (D + 2 fp32 a row) few.  (128 up to 4096: 62 us instead of 58.7 for the 32 contexts;
// 512 from 4096 on: 68; 256 throughout: 105 instead of 96 for the two long ones.)  Contexts of one leaf are finished here; others by qg_attn_merge_kernel.
#pragma once
#include "qg_attn_launch.cuh"
#include "qg_ptx.cuh"

namespace qg {

constexpr int kDecWarps = 8;
constexpr int kDecQueue = 4;       // leaves a warp may be ahead with its copies
constexpr float kLazy = 6.0f;      // a row's maximum moves when exceeded by 2^6

template <int KIND, int D, int NG>
struct Dec {
    static constexpr int REC = kv_record_bytes(KIND, D);
    static constexpr int SLOT = (REC + 127) & ~127;
    // Two CTAs per SM where the registers of one row group and a ring of at least three
    // records allow it; fp16 at D = 128 keeps 192 KB in flight in one.
    static constexpr int CTAS = NG == 1 && SLOT < 8192 ? 2 : 1;
    static constexpr int FIT = ((CTAS == 2 ? 113 : 227) * 1024 / kDecWarps - kDecQueue * 32) / (SLOT + 8);
    static constexpr int S = FIT > 8 ? 8 : FIT;  // ring slots of a warp
    static constexpr int SMEM = kDecWarps * (S * (SLOT + 8) + kDecQueue * 32);
    static_assert(S >= 3, "shared memory");
};

__host__ __device__ __forceinline__ int leaf_begin(int c)
{
    if (c < 16) return 64 * c;
    if (c < 24) return 1024 + 128 * (c - 16);
    if (c < 80) return 2048 + 256 * (c - 24);
    return 16384 + 512 * (c - 80);
}
__host__ __device__ __forceinline__ int leaf_of(int pos)
{
    if (pos < 1024) return pos >> 6;
    if (pos < 2048) return 16 + ((pos - 1024) >> 7);
    if (pos < 16384) return 24 + ((pos - 2048) >> 8);
    return 80 + ((pos - 16384) >> 9);
}
// First leaf of size class k (0..3), and one past the last of class 3.
__device__ __forceinline__ int class_begin(int k)
{
    return k == 0 ? 0 : k == 1 ? 16 : k == 2 ? 24 : k == 3 ? 80 : 0x7fffffff;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a request of this call is: its new tokens and its (cut) context.
struct Req {
    int q0, T, L;
    __device__ __forceinline__ int lo(const AttnParams &p) const  // first visible position
    {
        return p.window > 0 ? max(0, L - T - p.window + 1) : 0;
    }
};
__device__ __forceinline__ Req req_of(const AttnParams &p, int b)
{
    Req r;
    r.q0 = p.q_start[b];
    const int end = p.q_start[b + 1];
    r.T = end - r.q0;
    r.L = p.kv_len[b];
    bool bad = r.L > p.max_len || r.L < 0 || r.T > p.max_q || r.T < 0 || r.q0 < 0 || end > p.N;
    if (bad) {
        r.L = max(0, min(r.L, p.max_len));
        if (r.q0 < 0 || r.T < 0 || end > p.N)
            r.T = 0;
        else
            // the tail past max_q is dropped; the rest keeps its positions
            r.L = max(0, r.L - max(0, r.T - p.max_q)), r.T = min(r.T, p.max_q);
        atomicOr(p.err, kStatusRange);
    }
    return r;
}
__device__ __forceinline__ bool few_rows(const AttnParams &p, int T)
{
    return T > 0 && T * p.group <= p.few_max;
}

// log of sum 2^m.  The whole part of m goes into the sum first: added to log2(sum) it would
// take bits from it (m and log2(sum) have opposite signs where steps are small).
__device__ __forceinline__ float lse_of(float m, float sum)
{
    if (sum == 0.0f) return -INFINITY;
    const float whole = fminf(fmaxf(rintf(m), -60.0f), 60.0f);
    return logf(sum * exp2f(whole)) + (m - whole) * 0.6931471805599453f;
}

// Final result of one row: numbers d4 .. d4 + 3 and, once, the log of the sum.
__device__ __forceinline__ void store_row_out(const AttnParams &p, int64_t n, int h, int D, int d4,
                                              float4 a, float m, float sum)
{
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const __half2 x = __floats2half2_rn(a.x * inv, a.y * inv);
    const __half2 y = __floats2half2_rn(a.z * inv, a.w * inv);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t *>(&x);
    u.y = *reinterpret_cast<const uint32_t *>(&y);
    *reinterpret_cast<uint2 *>(p.out + n * p.os + (int64_t)h * D + d4) = u;
    if (p.lse && d4 == 0) p.lse[n * p.heads + h] = lse_of(m, sum);
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ float lds_f(uint32_t addr) { return __uint_as_float(lds32(addr)); }

// Multiplier bytes (one, or four at once) as mult_h2 wants them.  Q8's are 0..15: other bits can
// only come from rows past the context, where they must not make infinities (1152 * 127 would).
template <int KIND>
__device__ __forceinline__ uint32_t mult_byte(uint32_t m)
{
    return (KIND == KV_Q8 ? m & 0x0f0f0f0fu : m) ^ 0x80808080u;
}
// int8 multipliers a (low half) and b as fp16x2 (bytes already xored with 0x80).
__device__ __forceinline__ uint32_t mult_h2(uint32_t a, uint32_t b)
{
    return hsub2(0x64006400u | a | b << 16, 0x64806480u);
}
// Q8: code * mult = (1152 + code) * mult - 1152 * mult, exact (9 * 15 < 2^11).
// Q4: nibbles as fp16 subnormals n 2^-24: n 2^-24 * mult 2^8 - 8 mult 2^-16,
// exact, = (n - 8) mult 2^-16.
template <int KIND>
__device__ __forceinline__ uint32_t mult_scale(uint32_t m)
{
    return KIND == KV_Q8 ? m : hmul2(m, 0x5C005C00u);  // 2^8
}
template <int KIND>
__device__ __forceinline__ uint32_t mult_shift(uint32_t m)
{
    return KIND == KV_Q8 ? hmul2(m, 0xE480E480u) : hmul2(m, 0x88008800u);  // -1152, -2^-13
}

// Record row of m (or k) index i of a fragment: the order that keeps both the
// K and the V reads of the code rows free of bank conflicts.
__device__ __forceinline__ int frag_row(int i) { return i ^ ((i >> 1) & 1); }

template <int KIND, int D, int NG>
__global__ void __launch_bounds__(32 * kDecWarps, Dec<KIND, D, NG>::CTAS)
    qg_attn_decode_kernel(const __grid_constant__ AttnParams p)
{
    using C = Dec<KIND, D, NG>;
    constexpr int KS = D / 16;  // k steps of S, m tiles of O
    constexpr bool QUANT = KIND != KV_F16;
    extern __shared__ __align__(1024) uint8_t smem_dec[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(smem_dec) + warp * C::S * C::SLOT;
    int *const queue = reinterpret_cast<int *>(smem_dec + kDecWarps * C::S * C::SLOT) + warp * kDecQueue * 8;
    const uint32_t bars = smem_u32(smem_dec) + kDecWarps * (C::S * C::SLOT + kDecQueue * 32) + warp * C::S * 8;
    if (lane == 0) {
        for (int i = 0; i < C::S; ++i) mbar_init(bars + 8 * i, 1);
        mbar_fence_init();
    }
    __syncwarp();
    pdl_trigger();
    pdl_wait();

    // ---- the walk: leaves u, u + stride, ... of the list (size class from large to
    // small, request, leaf, part of the rows, head); 32 requests at a time, one per lane
    const int per_leaf = p.kv.heads * p.row_parts;
    int64_t u = (int64_t)warp * gridDim.x + blockIdx.x, base = 0;
    int wk = 3, wb = -32, n = 0, first = 0, cum = 0, c0 = 0, c1 = 0;
    Req wr = {0, 0, 0};
    auto window = [&](bool load) {  // 32 requests (read anew or not), and their leaves of class wk
        if (load) {
            wr.T = 0, c0 = c1 = 0;
            if (wb + lane < p.B) {
                wr = req_of(p, wb + lane);
                if (few_rows(p, wr.T)) c0 = leaf_of(wr.lo(p)), c1 = wr.L > 0 ? leaf_of(wr.L - 1) + 1 : c0 + 1;
            }
        }
        first = max(c0, class_begin(wk));
        n = max(0, min(c1, class_begin(wk + 1)) - first);
        cum = n;
        if (!__any_sync(~0u, n > 0)) return;  // (most classes of short contexts are empty)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, cum, o);
            if (lane >= o) cum += v;
        }
    };

    // ---- the copies: records ir .. ir1 - 1 of the walk's last leaf are still to be asked for
    int ir = 0, ir0 = 0, ir1 = 0, islot = 0, ahead = 0, pushed = 0, taken = 0;
    const uint8_t *isrc = nullptr;  // of record ir0 + lane (a leaf has at most 32)
    bool more = true, dead = false;
    auto fill = [&]() {
        while (ahead < C::S) {
            if (ir >= ir1) {
                if (!more || pushed - taken >= kDecQueue) return;
                int64_t rel;
                for (;;) {
                    const int total = __shfl_sync(~0u, cum, 31);
                    rel = u - base;
                    if (rel < (int64_t)total * per_leaf) break;
                    base += (int64_t)total * per_leaf;
                    const int before = wb;
                    wb += 32;
                    if (wb >= p.B && before >= 0) wb = 0, --wk;
                    if (wk < 0) {
                        more = false;
                        return;
                    }
                    window(wb != before);
                }
                u += (int64_t)gridDim.x * kDecWarps;
                // whose it is, and (a request's leaves x heads fit 32 bits) which of its
                const int src = __ffs(__ballot_sync(~0u, rel < (int64_t)cum * per_leaf)) - 1;
                const uint32_t own = (uint32_t)(rel - (int64_t)__shfl_sync(~0u, cum - n, src) * per_leaf);
                const uint32_t ci = own / (uint32_t)per_leaf, pk = own - ci * (uint32_t)per_leaf;
                const int part = NG > 1 && pk >= (uint32_t)p.kv.heads;
                const int row0 = part * 16, kh = (int)pk - part * p.kv.heads;
                const int c = __shfl_sync(~0u, first, src) + (int)ci;
                const int b = wb + src, L = __shfl_sync(~0u, wr.L, src), T = __shfl_sync(~0u, wr.T, src);
                const int q0 = __shfl_sync(~0u, wr.q0, src), lo = __shfl_sync(~0u, wr.lo(p), src);
                ir = ir0 = max(leaf_begin(c), lo) >> 4;
                ir1 = (min(leaf_begin(c + 1), L) + 15) >> 4;
                if (row0 >= T * p.group) ir1 = ir0;  // no rows in this part
                if (lane == 0) {
                    int4 *e = reinterpret_cast<int4 *>(queue + 8 * (pushed % kDecQueue));
                    e[0] = make_int4(b, c, kh | row0 << 16, L);
                    e[1] = make_int4(T, q0, ir0, ir1);
                }
                ++pushed;
                const int rec = ir0 + lane;
                if (rec < ir1) {
                    int64_t pg = p.table[b * p.table_stride + ((rec << 4) >> p.kv.page_shift)];
                    if (pg < 0 || pg >= (p.kv.slots >> p.kv.page_shift)) {
                        pg = 0;
                        atomicOr(p.err, kStatusRange);
                    }
                    isrc = p.kv.pool + (((pg * p.kv.heads + kh) << (p.kv.page_shift - 4)) +
                                        (rec & ((1 << (p.kv.page_shift - 4)) - 1))) * C::REC;
                }
                if (ahead > 0) return;  // the pages arrive while a record is worked on
                continue;
            }
            if (lane == ir - ir0) {
                mbar_arrive_expect_tx(bars + 8 * islot, C::REC);
                bulk_g2s(ring + islot * C::SLOT, isrc, C::REC, bars + 8 * islot);
            }
            ++ir, ++ahead;
            if (++islot == C::S) islot = 0;
        }
    };
    const int g = lane >> 2, t = lane & 3;
    int slot = 0, phase = 0;
    // (Q4: K's codes enter as (n - 8) 2^-20)
    const float sc2 = p.scale * 1.4426950408889634f * (KIND == KV_Q4 ? 1048576.0f : 1.0f);
    // token offset in a record of this lane's first score row (m index g; the other is 8 further)
    const int tok0 = QUANT ? frag_row(g) : g;
    // This lane's shared-memory offsets in a record.  fp16: ldmatrix rows of K and V (unit u of 64
    // numbers' line is xored in); codes: the K bytes of tok0 by block of 32 numbers (those of tok0 + 8
    // lie 8 rows on), and the V bytes of k indexes 2 t, 2 t + 1 (and 8 rows on).
    constexpr int R = kv_row_bytes(KIND, D);
    constexpr int NB = D / (KIND == KV_Q8 ? 8 : 16);  // V code bytes of this lane, per token
    const int ta = frag_row(2 * t), tb = frag_row(2 * t + 1);
    uint32_t k_at[KS / 2], v_at[2];
    if constexpr (QUANT) {
#pragma unroll
        for (int kb = 0; kb < KS / 2; ++kb)
            k_at[kb] = KIND == KV_Q8 ? kv_unit(KIND, D, tok0, 2 * kb + (t >> 1)) + 8 * (t & 1)
                                     : kv_unit(KIND, D, tok0, kb) + 4 * t;
        v_at[0] = kv_rows_at(KIND, D, 1) + kv_unit(KIND, D, ta, g * NB / 16) + (g * NB) % 16;
        v_at[1] = kv_rows_at(KIND, D, 1) + kv_unit(KIND, D, tb, g * NB / 16) + (g * NB) % 16;
    } else {
        const int kr = (lane & 7) + ((lane >> 3) & 1) * 8, vr = (lane & 7) + (lane >> 4) * 8;
        k_at[0] = kr * 128 + (((lane >> 4) ^ (kr & 7)) << 4);
        v_at[0] = kv_rows_at(KIND, D, 1) + vr * 128 + ((((lane >> 3) & 1) ^ (vr & 7)) << 4);
    }

    // The leaf in work: row r of the request is token r / group, head r % group of the kv head's (by a
    // product with 2^16 / group, exact below 64), and rows row0 .. row0 + 8 NG - 1 are this warp's.
    int b = 0, c = 0, kh = 0, row0 = 0, L = 0, T = 0, q0 = 0, rec = 0, r1 = 0, rows = 0, rf0 = 0, rf1 = 0, vlo = 0;
    int hi[NG][2], lo[NG][2];  // visible range [lo, hi) of this lane's rows row0 + 8 gi + 2 t + {0, 1}
    uint2 qf[NG][KS];          // q as B fragments (row g of each group of 8, the k order of the K fragments)
    float o[NG][KS][4], m[NG][2], l[NG][2];
    auto token_of = [&](int row) { return (int)((uint32_t)row * (uint32_t)p.group_inv >> 16); };
    bool open = false;
    // One turn: a record, or a leaf's end.  (Written so that the copies' code is there once: the first
    // run through a small call's code waits for its instructions.)
    for (;;) {
        fill();
        __syncwarp();
        if (!open) {
            if (taken == pushed) break;
            open = true;
            const int4 *const e = reinterpret_cast<const int4 *>(queue + 8 * (taken % kDecQueue));
            const int4 e0 = e[0], e1 = e[1];
            b = e0.x, c = e0.y, kh = e0.z & 0xffff, row0 = e0.z >> 16, L = e0.w;
            T = e1.x, q0 = e1.y, rec = e1.z, r1 = e1.w;
            rows = T * p.group;
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                const int row = row0 + 8 * gi + g, tr = token_of(row);
                const __half *q = p.q + (int64_t)(q0 + tr) * p.qs +
                                  (int64_t)(kh * p.group + row - tr * p.group) * D;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    qf[gi][ks] = make_uint2(0, 0);
                    if (row >= rows) continue;
                    if constexpr (KIND == KV_F16) {
                        const uint32_t *w = reinterpret_cast<const uint32_t *>(q + 16 * ks + 2 * t);
                        qf[gi][ks] = make_uint2(w[0], w[4]);
                    } else if constexpr (KIND == KV_Q8) {
                        qf[gi][ks] = *reinterpret_cast<const uint2 *>(q + 32 * (ks >> 1) + 8 * t + 4 * (ks & 1));
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(q + 16 * ks + 4 * t);
                        qf[gi][ks] = make_uint2(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632));
                    }
                }
            }

#pragma unroll
            for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int pos = L - T + token_of(min(row0 + 8 * gi + 2 * t + e2, rows - 1));
                    hi[gi][e2] = p.causal ? min(L, pos + 1) : L;
                    lo[gi][e2] = p.window > 0 ? pos - p.window + 1 : 0;
                }
            // records that every row sees whole, and the positions that any row sees
            rf0 = p.window > 0 ? (max(0, L - p.window) + 15) >> 4 : 0;
            rf1 = max(0, p.causal ? L - T + 1 : L) >> 4;
            vlo = p.window > 0 ? max(0, L - T - p.window + 1) : 0;
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
#pragma unroll
                for (int i = 0; i < KS; ++i) o[gi][i][0] = o[gi][i][1] = o[gi][i][2] = o[gi][i][3] = 0.0f;
                m[gi][0] = m[gi][1] = -INFINITY;
                l[gi][0] = l[gi][1] = 0.0f;
            }
        }

        if (rec < r1) {
            // (a copy that lands between two lanes' last polls: the lanes go on or give up together)
            const bool late = !mbar_wait(bars + 8 * slot, phase, 1u << 19);
            if (__any_sync(~0u, late)) {
                dead = true;
                break;
            }
            const uint32_t at = ring + slot * C::SLOT;
            const bool whole = rec >= rf0 && rec < rf1;
            const int j0 = rec * 16 + tok0;  // positions of this lane's score rows: j0, j0 + 8

            // Shared loads come before the arithmetic that hides them: K's, then V's while the
            // softmax runs.
            constexpr int KW = KIND == KV_Q8 ? 2 : 1, VW = NB / 4;
            constexpr int AHEAD = KS / 2;  // fp16: ldmatrix pairs in flight
            uint32_t kw[QUANT ? KS / 2 : 1][2][KW], vw[QUANT ? 4 : 1][VW];
            uint32_t fr[QUANT ? 1 : AHEAD + 1][8];
            float ks0 = sc2, ks1 = sc2, vs0 = 1.0f, vs1 = 1.0f, lg0 = 0.0f, lg1 = 0.0f;
            uint32_t km0 = 0, km1 = 0, ma = 0, mb = 0;
            auto load_v = [&]() {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a = at + v_at[k & 1] + (k >> 1) * 8 * R;
                    if constexpr (VW == 4) {
                        const uint4 v = lds128(a);
                        vw[k][0] = v.x, vw[k][1] = v.y, vw[k][2] = v.z, vw[k][3] = v.w;
                    } else if constexpr (VW == 2) {
                        const uint2 v = lds64(a);
                        vw[k][0] = v.x, vw[k][1] = v.y;
                    } else {
                        vw[k][0] = lds32(a);
                    }
                }
            };
            auto load_f = [&](uint32_t base, int i, uint32_t (&f)[8], bool trans) {  // units 4 i .. 4 i + 3
                const uint32_t a = at + (i >> 1) * 2048;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t(&r)[4] = *reinterpret_cast<uint32_t(*)[4]>(f + 4 * k);
                    const uint32_t x = a + (base ^ (((4 * i + 2 * k) & 7) << 4));
                    if (trans) ldsm4t(x, r);
                    else ldsm4(x, r);
                }
            };
            if constexpr (QUANT) {
#pragma unroll
                for (int kb = 0; kb < KS / 2; ++kb)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t a = at + k_at[kb] + k * 8 * R;
                        if constexpr (KIND == KV_Q8) {
                            const uint2 v = lds64(a);
                            kw[kb][k][0] = v.x, kw[kb][k][1] = v.y;
                        } else {
                            kw[kb][k][0] = lds32(a);
                        }
                    }
                uint32_t a = at + kv_mults_at(KIND, D, 0) + tok0 * (D / 32);
                if constexpr (D == 128)
                    km0 = lds32(a), km1 = lds32(a + 32);
                else
                    km0 = lds16(a), km1 = lds16(a + 16);
                a = at + kv_steps_at(KIND, D, 0) + 4 * tok0;
                ks0 = lds_f(a) * sc2, ks1 = lds_f(a + 32) * sc2;
                vs0 = lds_f(a + 64), vs1 = lds_f(a + 96);
                a = at + kv_mults_at(KIND, D, 1) + g / (256 / D);
                const uint32_t b0 = lds8(a + ta * (D / 32)), b1 = lds8(a + tb * (D / 32));
                const uint32_t b2 = lds8(a + (ta + 8) * (D / 32)), b3 = lds8(a + (tb + 8) * (D / 32));
                if constexpr (KIND == KV_Q4) load_v();
                ma = mult_h2(mult_byte<KIND>(b0) & 255, mult_byte<KIND>(b1) & 255);
                mb = mult_h2(mult_byte<KIND>(b2) & 255, mult_byte<KIND>(b3) & 255);
                km0 = mult_byte<KIND>(km0), km1 = mult_byte<KIND>(km1);
                if (!whole) {  // stale steps
                    if (j0 < vlo || j0 >= L) vs0 = 0.0f;
                    if (j0 + 8 < vlo || j0 + 8 >= L) vs1 = 0.0f;
                }
                // (steps of stored fp16 numbers are above 2^-40; zero rows weigh nothing)
                lg0 = fmaxf(__log2f(vs0), -40.0f), lg1 = fmaxf(__log2f(vs1), -40.0f);
            }
            uint32_t pf[NG][2];
            {
                // S^T.  fp16: even and odd k steps apart; codes: a sum for each block of
                // 32 numbers, which its multiplier then joins to the others in fp32
                float sa[NG][4], sb[NG][4];
                if constexpr (!QUANT) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) load_f(k_at[0], i, fr[i], false);
                }
#pragma unroll
                for (int kb = 0; kb < KS / 2; ++kb) {
                    if constexpr (!QUANT) {
                        if (kb + AHEAD < KS / 2) load_f(k_at[0], kb + AHEAD, fr[(kb + AHEAD) % (AHEAD + 1)], false);
                        uint32_t(&f)[8] = fr[kb % (AHEAD + 1)];
#pragma unroll
                        for (int gi = 0; gi < NG; ++gi) {
                            const uint2 qa = qf[gi][2 * kb], qb = qf[gi][2 * kb + 1];
                            if (kb == 0) {
                                mma16816_zc(sa[gi], f[0], f[1], f[2], f[3], qa.x, qa.y);
                                mma16816_zc(sb[gi], f[4], f[5], f[6], f[7], qb.x, qb.y);
                            } else {
                                mma16816(sa[gi], f[0], f[1], f[2], f[3], qa.x, qa.y);
                                mma16816(sb[gi], f[4], f[5], f[6], f[7], qb.x, qb.y);
                            }
                        }
                    } else {
                        uint32_t a[8];  // A fragments of k steps 2 kb, 2 kb + 1: the codes, exact
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if constexpr (KIND == KV_Q8) {
                                const uint32_t x = kw[kb][k][0] ^ 0x80808080u, y = kw[kb][k][1] ^ 0x80808080u;
                                a[k] = hsub2(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
                                a[k + 2] = hsub2(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
                                a[k + 4] = hsub2(__byte_perm(y, 0x64646464u, 0x4140), 0x64806480u);
                                a[k + 6] = hsub2(__byte_perm(y, 0x64646464u, 0x4342), 0x64806480u);
                            } else {
                                // (n - 8) 2^-20: low nibbles are n 2^-24 and times 16, high ones lie as
                                // 16 n 2^-24.  (Both as they lie, with q / 16 for the high ones, took
                                // bits from a q below 2^-10.)
                                const uint32_t x = kw[kb][k][0], y = x >> 8;
                                a[k] = hfma2(x & 0x000f000fu, 0x4C004C00u, 0x80808080u);
                                a[k + 2] = hfma2(y & 0x000f000fu, 0x4C004C00u, 0x80808080u);
                                a[k + 4] = hsub2(x & 0x00f000f0u, 0x00800080u);
                                a[k + 6] = hsub2(y & 0x00f000f0u, 0x00800080u);
                            }
                        }
                        // 2^23 + (m + 128) as bits, less that
                        const float m0 = __uint_as_float(__byte_perm(km0, 0x4B000000u, 0x7540 | kb)) - 8388736.0f;
                        const float m1 = __uint_as_float(__byte_perm(km1, 0x4B000000u, 0x7540 | kb)) - 8388736.0f;
#pragma unroll
                        for (int gi = 0; gi < NG; ++gi) {
                            const uint2 qa = qf[gi][2 * kb], qb = qf[gi][2 * kb + 1];
                            float(&x)[4] = sa[gi], c4[4];
                            mma16816_zc(c4, a[0], a[1], a[2], a[3], qa.x, qa.y);
                            mma16816(c4, a[4], a[5], a[6], a[7], qb.x, qb.y);
                            if (kb == 0) {
                                x[0] = c4[0] * m0, x[1] = c4[1] * m0, x[2] = c4[2] * m1, x[3] = c4[3] * m1;
                            } else {
                                x[0] = fmaf(c4[0], m0, x[0]), x[1] = fmaf(c4[1], m0, x[1]);
                                x[2] = fmaf(c4[2], m1, x[2]), x[3] = fmaf(c4[3], m1, x[3]);
                            }
                        }
                    }
                }
                {  // V's loads fly under the softmax
                    if constexpr (KIND == KV_Q8) load_v();
                    if constexpr (!QUANT) {
#pragma unroll
                        for (int i = 0; i < AHEAD; ++i) load_f(v_at[0], i, fr[i], true);
                    }
                }
                bool up = false;
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    float(&x)[4] = sa[gi];
                    if constexpr (!QUANT) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] += sb[gi][i];
                    }
                    x[0] *= ks0, x[1] *= ks0, x[2] *= ks1, x[3] *= ks1;
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (j0 < lo[gi][e] || j0 >= hi[gi][e]) x[e] = -INFINITY;
                            if (j0 + 8 < lo[gi][e] || j0 + 8 >= hi[gi][e]) x[2 + e] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) up |= fmaxf(x[e] + lg0, x[2 + e] + lg1) > m[gi][e] + kLazy;
                }
                if (__any_sync(~0u, up)) {
                    // rows whose own maximum was exceeded move to the new one
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(sa[gi][e] + lg0, sa[gi][2 + e] + lg1);
                            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                            if (mx > m[gi][e] + kLazy) {
                                const float al = m[gi][e] == -INFINITY ? 1.0f : ex2(m[gi][e] - mx);
                                m[gi][e] = mx;
                                l[gi][e] *= al;
#pragma unroll
                                for (int i = 0; i < KS; ++i) o[gi][i][e] *= al, o[gi][i][2 + e] *= al;
                            }
                        }
                }
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    const float m0 = m[gi][0] == -INFINITY ? 0.0f : m[gi][0];
                    const float m1 = m[gi][1] == -INFINITY ? 0.0f : m[gi][1];
                    const float p0 = ex2(sa[gi][0] - m0), p1 = ex2(sa[gi][1] - m1);
                    const float p2 = ex2(sa[gi][2] - m0), p3 = ex2(sa[gi][3] - m1);
                    l[gi][0] += p0 + p2;
                    l[gi][1] += p1 + p3;
                    // the one rounding to 16 bits between scores and result
                    pf[gi][0] = transpose8(pack_h2(p0 * vs0, p1 * vs0));
                    pf[gi][1] = transpose8(pack_h2(p2 * vs1, p3 * vs1));
                }
            }

            // O^T += V^T P^T
            if constexpr (!QUANT) {
                uint32_t k01 = ~0u, k89 = ~0u;  // keeps of token pairs 2 t, 2 t + 1 and + 8
                if (!whole) {
                    const int j = rec * 16 + 2 * t;
                    auto keep = [&](int jj) {
                        return (jj >= vlo && jj < L ? 0xffffu : 0u) |
                               (jj + 1 >= vlo && jj + 1 < L ? 0xffff0000u : 0u);
                    };
                    k01 = keep(j), k89 = keep(j + 8);
                }
#pragma unroll
                for (int i = 0; i < KS / 2; ++i) {
                    if (i + AHEAD < KS / 2) load_f(v_at[0], i + AHEAD, fr[(i + AHEAD) % (AHEAD + 1)], true);
                    uint32_t(&f)[8] = fr[i % (AHEAD + 1)];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t *a = f + 4 * k;
                        if (!whole) a[0] &= k01, a[1] &= k01, a[2] &= k89, a[3] &= k89;
#pragma unroll
                        for (int gi = 0; gi < NG; ++gi)
                            mma16816(o[gi][2 * i + k], a[0], a[1], a[2], a[3], pf[gi][0], pf[gi][1]);
                    }
                }
            } else {
                const uint32_t fa = mult_scale<KIND>(ma), fb = mult_scale<KIND>(mb);
                const uint32_t ha = mult_shift<KIND>(ma), hb = mult_shift<KIND>(mb);
                if constexpr (KIND == KV_Q8) {
#pragma unroll
                    for (int q = 0; q < VW; ++q) {  // m tiles 2 q, 2 q + 1: numbers 4 q .. 4 q + 3
                        const uint32_t x0 = vw[0][q] ^ 0x80808080u, x1 = vw[1][q] ^ 0x80808080u;
                        const uint32_t y0 = vw[2][q] ^ 0x80808080u, y1 = vw[3][q] ^ 0x80808080u;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x = __byte_perm(x0, x1, e ? 0x7362 : 0x5140);
                            const uint32_t y = __byte_perm(y0, y1, e ? 0x7362 : 0x5140);
                            const uint32_t a0 = hfma2(__byte_perm(x, 0x64646464u, 0x4140), fa, ha);
                            const uint32_t a1 = hfma2(__byte_perm(x, 0x64646464u, 0x4342), fa, ha);
                            const uint32_t a2 = hfma2(__byte_perm(y, 0x64646464u, 0x4140), fb, hb);
                            const uint32_t a3 = hfma2(__byte_perm(y, 0x64646464u, 0x4342), fb, hb);
#pragma unroll
                            for (int gi = 0; gi < NG; ++gi)
                                mma16816(o[gi][2 * q + e], a0, a1, a2, a3, pf[gi][0], pf[gi][1]);
                        }
                    }
                } else {
                    const uint32_t fah = hmul2(fa, 0x2C002C00u), fbh = hmul2(fb, 0x2C002C00u);  // / 16
#pragma unroll
                    for (int i = 0; i < KS; ++i) {  // byte i: low nibbles row g, high nibbles row g + 8
                        const uint32_t sel = (i & 3) * 0x1111u + 0x4400u;
                        const uint32_t x = __byte_perm(vw[0][i / 4], vw[1][i / 4], sel);
                        const uint32_t y = __byte_perm(vw[2][i / 4], vw[3][i / 4], sel);
                        const uint32_t a0 = hfma2(x & 0x000f000fu, fa, ha);
                        const uint32_t a1 = hfma2(x & 0x00f000f0u, fah, ha);
                        const uint32_t a2 = hfma2(y & 0x000f000fu, fb, hb);
                        const uint32_t a3 = hfma2(y & 0x00f000f0u, fbh, hb);
#pragma unroll
                        for (int gi = 0; gi < NG; ++gi)
                            mma16816(o[gi][i], a0, a1, a2, a3, pf[gi][0], pf[gi][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the record
            if (++slot == C::S) slot = 0, phase ^= 1;
            --ahead;
            ++rec;
            continue;
        }
        ++taken;
        open = false;

        // ---- the leaf's rows
        const bool only = leaf_of(vlo) >= leaf_of(max(L, 1) - 1);  // the context's one leaf
        constexpr float kOut = KIND == KV_Q4 ? 65536.0f : 1.0f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
                float sum = l[gi][e2];
                sum += __shfl_xor_sync(~0u, sum, 4);
                sum += __shfl_xor_sync(~0u, sum, 8);
                sum += __shfl_xor_sync(~0u, sum, 16);
                const int row = row0 + 8 * gi + 2 * t + e2;
                if (row >= rows) continue;
                const int tr = token_of(row), h = kh * p.group + row - tr * p.group;
                const int64_t n0 = q0 + tr;
                const int64_t at = ((int64_t)(q0 * p.row_q + b * p.row_b + tr) * p.heads + h) * p.few_leaves + c;
                const float mx = m[gi][e2];
                if (g == 0) {
                    if (!only)
                        p.ws_ml[at] = make_float2(mx, sum);
                    else if (p.lse)
                        p.lse[n0 * p.heads + h] = lse_of(mx, sum);
                }
                const float f = only ? (sum == 0.0f ? 0.0f : kOut / sum) : kOut;
                // this lane's numbers of the row: runs of four where the codes' order gives them
                __half *const oh = p.out + n0 * p.os + (int64_t)h * D;
                float *const of = p.ws_o + at * D;
                if constexpr (KIND == KV_F16) {
#pragma unroll
                    for (int i = 0; i < KS; ++i)
#pragma unroll
                        for (int u8 = 0; u8 < 2; ++u8) {
                            const int d = 16 * i + 8 * u8 + g;
                            const float v = o[gi][i][2 * u8 + e2] * f;
                            if (only) oh[d] = __float2half_rn(v);
                            else of[d] = v;
                        }
                } else {
                    constexpr int RUNS = D / 32;  // of this lane's D / 8 numbers
#pragma unroll
                    for (int q = 0; q < RUNS; ++q) {
                        float v[4];
                        int d;
                        if constexpr (KIND == KV_Q8) {
                            d = (D / 8) * g + 4 * q;
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] = o[gi][2 * q + (i >> 1)][2 * (i & 1) + e2] * f;
                        } else {
                            constexpr int HALF = RUNS / 2;  // runs of low, then of high nibbles
                            d = 32 * (g / (256 / D)) + 16 * (q / HALF) + (D / 16) * (g % (256 / D)) + 4 * (q % HALF);
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] = o[gi][4 * (q % HALF) + i][2 * (q / HALF) + e2] * f;
                        }
                        if (only)
                            *reinterpret_cast<uint2 *>(oh + d) = make_uint2(pack_h2(v[0], v[1]), pack_h2(v[2], v[3]));
                        else
                            *reinterpret_cast<float4 *>(of + d) = make_float4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
    }
    if (dead) {
        // a copy did not arrive in time: those in flight get the same time again
        if (lane == 0) atomicOr(p.err, 1u);
        for (; ahead > 0; --ahead) {
            mbar_wait(bars + 8 * slot, phase, 1u << 19);
            if (++slot == C::S) slot = 0, phase ^= 1;
        }
    }
}

}  // namespace qg
