// Attention of many rows: chunks and prompts, requests of more than kDecRows rows
// (new tokens x heads of a kv head), on the tensor cores (tcgen05, tensor memory).
//
// A CTA takes up to 256 rows of one (request, kv head): two tiles A and B of 128 rows, a row
// being a (token, head of the group) pair, so the heads of a group share every K and V tile.
// It goes over the visible keys in tiles of 128:
//   S = Q K^T    tcgen05.mma, Q and K from shared memory, S (128 x 128 fp32) in tensor memory
//   P = 2^(S scale - m), one thread per row, fp16, back into tensor memory
//   O += P V     tcgen05.mma, P from tensor memory, V from shared memory
// Two softmax warpgroups (one per tile), one MMA thread, and loaders.  The MMA thread's order is
//   Q_A K(i + 1), P_A V(i), Q_B K(i + 1), P_B V(i)
// so that S of the next key tile is ready when a softmax ends: the softmaxes (about 1650 cycles a
// key tile, 1000 of them for the 16384 exponentials) run under the products of 4 x 512 cycles at
// D = 128.  Measured 2640 cycles a key tile, 352-394 us for a prompt of 8192 tokens and 32 heads
// (by the card and its power): 1.40-1.56 PFLOP/s, tensor pipe 67 % busy; the rest is the waits between the products and, for
// a CTA, 7000 cycles before its first product and 4700 after its last.  At D = 64 the softmaxes
// bound it (2440 with windows; an S for each tile, which fits there: 2 % less).
// Tensor memory holds it because a softmax takes S into registers at once: one S for
// both tiles (128 columns), P_A and P_B (64 each), O_A and O_B (128 each).  (With P in S's place
// a tile's chain of products and softmax is serial: 3100 cycles a key tile, 428 us for the
// 8192-token prompt.)  The output is rescaled only when a row's maximum grows by more than
// 2^kLazy; the softmax threads do it themselves, when the previous product has ended.
//
// The cache's fp16 records are stored as 128-byte-swizzled pieces, so bulk copies put them into
// shared memory as operands (K: K-major; V: MN-major, both [64 numbers][128 tokens][128 B]).
// Codes are decoded by a warpgroup of loaders into the same tiles as mult * code (exact); K's
// steps multiply the scores of their column, V's steps enter the exponent as log2(step) and
// are taken out of the sums of p again.  There the softmax is the longest part (three numbers
// from shared memory for every column), so it is written for issue slots and code size instead:
// it goes over S in tensor memory twice, 32 columns at a time, each tile with an S of its own that
// P overwrites.  (Unrolled with S in registers as for fp16, its warps waited for instructions
// more than for anything else: 7000 cycles a key tile.)
//
// Few tiles and long contexts: the keys are cut into p.splits parts, each a CTA, joined by
// qg_attn_join_kernel.
#pragma once
#include "qg_attn_decode.cuh"

namespace qg {

// Polls of a wait before it gives up: each suspends for up to a few microseconds.
constexpr uint32_t kWaitLimit = 1u << 19;

template <int KIND, int D>
struct Chunk {
    static constexpr bool QUANT = KIND != KV_F16;
    static constexpr int TILE = 128 * D * 2;              // bytes of a Q, K or V tile
    static constexpr int HALVES = D / 64;
    static constexpr int NS = QUANT ? 3 : D == 64 ? 8 : 5;  // K / V slots, in turn
    // codes: [key tile mod 4][ck, lg, rv][128], the rows as they are stored (three K or V parts of
    // a key tile), and the steps and multipliers of four key tiles.  (What belongs to key tile
    // i is written again with K(i + 4), once V(i + 1) has been used: A and B are past tile i.)
    static constexpr int SCALES = QUANT ? 4 * 3 * 512 : 0;
    static constexpr int PARTS = 3, PART = QUANT ? 128 * kv_row_bytes(KIND, D) : 0;
    static constexpr int SMALL = QUANT ? kv_record_bytes(KIND, D) - 32 * kv_row_bytes(KIND, D) : 0;  // of a record
    static constexpr int STAGE = PARTS * PART + 4 * 8 * SMALL;
    static constexpr int BARS = 512;
    static constexpr int SMEM = 2 * TILE + NS * TILE + SCALES + STAGE + BARS;
    // warps: 0-3, 4-7 softmax of A and B; 8 MMA; 9 (fp16: 9 K, 10 V) copies;
    // 12-15 decoders (codes)
    static constexpr int WARPS = QUANT ? 16 : 12;
    // fp16, registers: 12 x 32 x 168 = 8 x 32 x 208 + 4 x 32 x 88
    static constexpr int REGS_HI = 208, REGS_LO = 88;
    // tensor memory: S and P of tile w; O of tile w is at 256 + 128 w.  fp16: one S, P_A, P_B;
    // codes: S_A, S_B, and P in S's place.
    __host__ __device__ static constexpr uint32_t S_AT(int w) { return QUANT ? 128u * w : 0u; }
    __host__ __device__ static constexpr uint32_t P_AT(int w) { return QUANT ? 128u * w : 128u + 64u * w; }
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Shared-memory descriptors with the 128-byte swizzle (bits 61-63 = 2): K-major operands have
// 8-row groups 1024 B apart (one 64-number half at a time); MN-major operands have the next 64
// numbers `lbo` bytes on and the next 8 k rows 1024 B on.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t pk2(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void upk2(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// A descriptor `bytes` further on (addresses are in its low word and stay below 2^18 bytes).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes)
{
    return (d & 0xffffffff00000000ull) | ((uint32_t)d + (bytes >> 4));
}
// S = Q K^T of one tile (KS MMAs of 16 numbers, four to a 64-number half, 16 KB on).
template <int KS>
__device__ __forceinline__ void batch_qk(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc, uint32_t done)
{
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const uint32_t at = (i >> 2) * 16384 + (i & 3) * 32;
        tc_mma_ss(d, desc_at(q, at), desc_at(k, at), idesc, i > 0);
    }
    tc_commit(done);
}
// O += P V of one tile (8 MMAs of 16 keys, P from tensor memory).
__device__ __forceinline__ void batch_pv(uint32_t d, uint32_t pt, uint64_t v, uint32_t idesc, bool add, uint32_t done)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) tc_mma(d, pt + 8 * i, desc_at(v, i * 2048), idesc, add || i > 0);
    tc_commit(done);
}

// Everything the MMA thread does for one or two tiles and nt key tiles.  Each batch waits for what
// it needs as it comes to it, the tile from the cache first: its wait is over long before.
// (Asking for the next batch's barriers in the middle of a batch, to hide a wait's latency, made
// a key tile take 2890 cycles instead of 2500: the question queues behind the MMAs.)
template <int KIND, int D, bool TWO, class Wait>
__device__ __forceinline__ void mma_thread(uint32_t tmem, uint32_t sq, uint32_t skv, uint32_t b_full,
                                           uint32_t b_empty, uint32_t b_q, uint32_t b_s, uint32_t b_sf,
                                           uint32_t b_p, uint32_t b_o, int nt, Wait &wait)
{
    using C = Chunk<KIND, D>;
    constexpr int NS = C::NS, TILE = C::TILE, KS = D / 16;
    constexpr bool ONE_S = !C::QUANT;  // one S for both tiles
    constexpr uint32_t kS = tc_idesc_f16(128);
    constexpr uint32_t kO = tc_idesc_f16(D) | (1u << 16);  // V is MN-major
    const uint64_t q[2] = {desc_sw128(sq, 0), desc_sw128(sq + TILE, 0)};
    const uint64_t dk = desc_sw128(skv, 0), dv = desc_sw128(skv, 16384);
    // K(it + 1) is number 2 it + 1 of the ring, V(it) number 2 it + 2
    uint32_t ks = 1, kp = 0, vs = 2, vp = 0;
    wait(b_full, 0);
#pragma unroll
    for (int w = 0; w <= (int)TWO; ++w) {
        wait(b_q + 8 * w, 0);
        if (ONE_S && w) wait(b_sf, 0);  // S of A has been taken
        tc_fence_after();
        batch_qk<KS>(tmem + C::S_AT(w), q[w], dk, kS, b_s + 8 * w);
    }
    tc_commit(b_empty);
#pragma unroll 1
    for (int it = 0; it < nt; ++it) {
        const bool more = it + 1 < nt;
        const uint32_t par = it & 1;
        const uint64_t k = desc_at(dk, ks * TILE), v = desc_at(dv, vs * TILE);
        if (more) wait(b_full + 8 * ks, kp);
        if (!ONE_S) wait(b_full + 8 * vs, vp);
#pragma unroll
        for (int w = 0; w <= (int)TWO; ++w) {
            auto qk = [&]() {
                if (more) {
                    // S is free: of B(it) for A, of A(it + 1) for B (alone: of A(it))
                    if (ONE_S) wait(b_sf, !TWO ? par : w ? 0u : 1u);
                    tc_fence_after();
                    batch_qk<KS>(tmem + C::S_AT(w), q[w], k, kS, b_s + 8 * w);
                    if (w == (int)TWO) tc_commit(b_empty + 8 * ks);
                }
            };
            if (ONE_S) {
                qk();
                if (w == 0) wait(b_full + 8 * vs, vp);
            }
            wait(b_p + 8 * w, par);
            tc_fence_after();
            batch_pv(tmem + 256 + 128 * w, tmem + C::P_AT(w), v, kO, it > 0, b_o + 8 * w);
            if (w == (int)TWO) tc_commit(b_empty + 8 * vs);
            if (!ONE_S) qk();  // P was in S's place
        }
        ks += 2, vs += 2;
        if (ks >= NS) ks -= NS, kp ^= 1;
        if (vs >= NS) vs -= NS, vp ^= 1;
    }
}

// One thread of a converged warp, known to the compiler as such: what it feeds to the MMAs stays
// in uniform registers (chosen by lane == 0 each MMA cost about 100 cycles to issue).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

template <int N>
__device__ __forceinline__ void reg_grow()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_shrink()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

template <int KIND, int D>
__global__ void __launch_bounds__(32 * Chunk<KIND, D>::WARPS, 1)
    qg_attn_chunk_kernel(const __grid_constant__ AttnParams p)
{
    using C = Chunk<KIND, D>;
    constexpr bool QUANT = C::QUANT;
    constexpr int NS = C::NS, TILE = C::TILE;
    extern __shared__ __align__(1024) uint8_t smem_chunk[];
    const uint32_t sq = smem_u32(smem_chunk), skv = sq + 2 * TILE;
    float *const scales = reinterpret_cast<float *>(smem_chunk + (2 + NS) * TILE);
    const uint32_t stage = sq + (2 + NS) * TILE + C::SCALES, small = stage + C::PARTS * C::PART;
    const uint32_t bars = stage + C::STAGE;
    const uint32_t b_full = bars, b_empty = bars + 64, b_q = bars + 128, b_s = bars + 144,
                   b_p = bars + 160, b_o = bars + 176, b_sc = bars + 192, b_end = bars + 224, b_sf = bars + 232, tm_at = bars + 240,
                   b_in = bars + 256, b_out = bars + 288;
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(b_full + 8 * i, QUANT ? 4 : 32);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_q + 8 * i, 128);
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_p + 8 * i, 4);
            mbar_init(b_o + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(b_sc + 8 * i, 4);
        for (int i = 0; i < C::PARTS; ++i) {
            mbar_init(b_in + 8 * i, 8);
            mbar_init(b_out + 8 * i, 4);
        }
        mbar_init(b_sf, 4);
        mbar_init(b_end, 1);
        mbar_fence_init();
    }
    if (warp == 8) tmem_alloc(tm_at, 512);
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tm_at));
    tmem = __shfl_sync(~0u, tmem, 0);
    pdl_wait();

    // ---- which rows: blockIdx.x = (tile pair, part of the keys, head), the pairs of a request
    // from the last (most keys) to the first
    const int TT = 128 / p.group;  // tokens of a tile
    int b = -1, pair = 0;
    Req r = {0, 0, 0};
    const int kh = blockIdx.x % p.kv.heads, part = blockIdx.x / p.kv.heads % p.splits;
    {
        int left = blockIdx.x / p.kv.heads / p.splits;
        for (int b0 = 0; b0 < p.B && b < 0; b0 += 32) {
            Req q = {0, 0, 0};
            int n = 0;
            if (b0 + lane < p.B) {
                q = req_of(p, b0 + lane);
                if (q.T > 0 && !few_rows(p, q.T)) n = (q.T + 2 * TT - 1) / (2 * TT);
            }
            int cum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(~0u, cum, o);
                if (lane >= o) cum += v;
            }
            const uint32_t in = __ballot_sync(~0u, left < cum);
            if (in) {
                const int src = __ffs(in) - 1;
                b = b0 + src;
                pair = __shfl_sync(~0u, cum - 1 - left, src);  // from the last to the first
                r.q0 = __shfl_sync(~0u, q.q0, src);
                r.T = __shfl_sync(~0u, q.T, src);
                r.L = __shfl_sync(~0u, q.L, src);
            } else {
                left -= __shfl_sync(~0u, cum, 31);
            }
        }
    }
    const int t0 = pair * 2 * TT;                          // first token of the pair
    const int t1 = min(r.T, t0 + 2 * TT);                  // past the last
    const bool two = t1 - t0 > TT;                         // tile B has rows
    const int p0 = r.L - r.T + t0, p1 = r.L - r.T + t1;    // their positions
    const int hi_u = max(0, p.causal ? min(r.L, p1) : r.L);
    const int lo_u = p.window > 0 ? max(0, p0 - p.window + 1) : 0;
    int j0 = lo_u >> 7, j1 = (hi_u + 127) >> 7;
    if (b < 0 || hi_u <= lo_u) j1 = j0;
    {
        const int n = j1 - j0;
        j1 = j0 + (int)((int64_t)n * (part + 1) / p.splits);
        j0 += (int)((int64_t)n * part / p.splits);
    }
    const int nt = j1 - j0;  // key tiles of this CTA
    // After a wait that ran out, the thread's further waits return at once.
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, kWaitLimit)) {
            dead = true;
            atomicOr(p.err, 1u);
        }
    };

    if (warp < 8) {
        if constexpr (!QUANT) reg_grow<C::REGS_HI>();
        // ---- softmax of tile w: row `row` = token t, head kh * group + hg
        const int w = warp >> 2, row = threadIdx.x & 127;
        const int tl = row / p.group, t = t0 + w * TT + tl;
        const bool live = b >= 0 && tl < TT && t < t1;
        const int h = kh * p.group + row - tl * p.group;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // tensor-memory lanes 32 (warp mod 4) ..
        const uint32_t ts = tmem + lanes + C::S_AT(w), tp = tmem + lanes + C::P_AT(w);
        const uint32_t to = tmem + lanes + 256 + 128 * w;
        if (b >= 0 && (w == 0 || two)) {
            // Q into shared memory as a swizzled K-major operand, each warp its own 32 rows, whole
            // rows at a time (one thread per row: 10000 cycles); a negative scale turns its signs
            const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;
            const __half *own = live ? p.q + (int64_t)(r.q0 + t) * p.qs + (int64_t)h * D : nullptr;
            constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows of a load
            uint4 v[LPR];
#pragma unroll
            for (int i = 0; i < LPR; ++i) {
                const __half *q = reinterpret_cast<const __half *>(
                    __shfl_sync(~0u, (unsigned long long)own, i * RPI + lane / LPR));
                v[i] = q ? *reinterpret_cast<const uint4 *>(q + 8 * (lane % LPR)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < LPR; ++i) {
                const int rw = (row & 96) + i * RPI + lane / LPR, u = lane % LPR;
                const uint32_t at = sq + w * TILE + (u >> 3) * 16384 + rw * 128 + (((u & 7) ^ (rw & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[i].x ^ flip),
                             "r"(v[i].y ^ flip), "r"(v[i].z ^ flip), "r"(v[i].w ^ flip)
                             : "memory");
            }
            fence_proxy_async_smem();
            mbar_arrive(b_q + 8 * w);
        }
        const int pos = r.L - r.T + t;
        const int hi = live && p.causal ? min(r.L, pos + 1) : r.L;
        const int lo = live && p.window > 0 ? pos - p.window + 1 : 0;
        // (a scale of zero still needs -inf for hidden keys)
        const float sc2 = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-30f);
        float m = -INFINITY;
        uint64_t l2[4];  // the sum of p, in eight parts
#pragma unroll
        for (int i = 0; i < 4; ++i) l2[i] = pk2(0.0f, 0.0f);
        if (w == 1 && !two) goto done;
        {
            // this row's running maximum moves to `top` (score and, for codes, log2 of V's step)
            auto move_to = [&](float top, int it) {
                const bool up = top > m + kLazy;
                if (!__any_sync(~0u, up)) return;
                const float al = up && m != -INFINITY ? ex2(m - top) : 1.0f;
                if (up) m = top;
                const uint64_t al2 = pk2(al, al);
#pragma unroll
                for (int i = 0; i < 4; ++i) asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(l2[i]) : "l"(al2));
                if (it == 0) return;
                wait(b_o + 8 * w, (it - 1) & 1);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                    tmem_st32(to + 32 * c, o);
                }
            };
            auto p_done = [&]() {
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p + 8 * w);
            };
            for (int it = 0; it < nt; ++it) {
                wait(b_s + 8 * w, it & 1);
                tc_fence_after();
                const int jb = (j0 + it) << 7;
                const bool all = __all_sync(~0u, jb >= lo && jb + 128 <= hi);
                if constexpr (!QUANT) {
                    float s[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tmem_ld32(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
                    tc_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_sf);  // S may be overwritten
                    if (!all) {  // (one compare a number and end: most tiles are cut at one end)
                        const int from = lo - jb, to = hi - jb;
                        if (__any_sync(~0u, to < 128)) {
#pragma unroll
                            for (int i = 0; i < 128; ++i) s[i] = i < to ? s[i] : -INFINITY;
                        }
                        if (__any_sync(~0u, from > 0)) {
#pragma unroll
                            for (int i = 0; i < 128; ++i) s[i] = i >= from ? s[i] : -INFINITY;
                        }
                    }
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int i = 4; i < 124; i += 8) {
                        mx[0] = max3(mx[0], s[i], s[i + 4]), mx[1] = max3(mx[1], s[i + 1], s[i + 5]);
                        mx[2] = max3(mx[2], s[i + 2], s[i + 6]), mx[3] = max3(mx[3], s[i + 3], s[i + 7]);
                    }
                    mx[0] = max3(mx[0], s[124], s[125]), mx[1] = max3(mx[1], s[126], s[127]);
                    move_to(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc2, it);
                    const float mm = m == -INFINITY ? 0.0f : m;
                    const uint64_t nm2 = pk2(-mm, -mm), sc22 = pk2(sc2, sc2);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t ph[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int k = 64 * c + 2 * i;
                            float x, y;
                            upk2(fma2(pk2(s[k], s[k + 1]), sc22, nm2), x, y);
                            x = ex2(x), y = ex2(y);
                            l2[i & 3] = add2(l2[i & 3], pk2(x, y));
                            ph[i] = pack_h2(x, y);  // the one rounding to 16 bits between scores and result
                        }
                        if (c == 0 && it > 0) {
                            wait(b_o + 8 * w, (it - 1) & 1);  // P(it - 1) has been used
                            tc_fence_after();
                        }
                        tmem_st32(tp + 32 * c, ph);
                    }
                    p_done();
                } else {
                    const float *const sc = scales + (it & 3) * 384;
                    wait(b_sc + 8 * (it & 3), (it >> 2) & 1);
                    // scores with their steps, back in their place
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        float s[32];
                        tmem_ld32(ts + c, *reinterpret_cast<uint32_t(*)[32]>(s));
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 ck = *reinterpret_cast<const float4 *>(sc + c + i);
                            const float4 lg = *reinterpret_cast<const float4 *>(sc + 128 + c + i);
                            upk2(fma2(pk2(s[i], s[i + 1]), pk2(ck.x, ck.y), pk2(lg.x, lg.y)), s[i], s[i + 1]);
                            upk2(fma2(pk2(s[i + 2], s[i + 3]), pk2(ck.z, ck.w), pk2(lg.z, lg.w)), s[i + 2], s[i + 3]);
                        }
                        if (!all) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) s[i] = i < hi - jb - c && i >= lo - jb - c ? s[i] : -INFINITY;
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], s[i + k], s[i + 4 + k]);
                        tmem_st32(ts + c, *reinterpret_cast<uint32_t(*)[32]>(s));
                    }
                    move_to(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), it);
                    const float mm = m == -INFINITY ? 0.0f : m;
                    const uint64_t nm2 = pk2(-mm, -mm);
                    tc_wait_st();
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        float s[32];
                        uint32_t ph[16];
                        tmem_ld32(ts + c, *reinterpret_cast<uint32_t(*)[32]>(s));
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 rv = *reinterpret_cast<const float4 *>(sc + 256 + c + i);
#pragma unroll
                            for (int k = 0; k < 4; k += 2) {
                                float x, y;
                                upk2(add2(pk2(s[i + k], s[i + k + 1]), nm2), x, y);
                                x = ex2(x), y = ex2(y);
                                uint64_t &l = l2[(i / 4 & 1) * 2 + k / 2];
                                l = fma2(pk2(x, y), k ? pk2(rv.z, rv.w) : pk2(rv.x, rv.y), l);
                                ph[(i + k) / 2] = pack_h2(x, y);
                            }
                        }
                        tmem_st16(tp + c / 2, ph);  // (below the columns still to be read)
                    }
                    p_done();
                }
            }
        }
        {
            float la, lb;
            upk2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])), la, lb);
            const float sum = la + lb;
            if (nt > 0) {
                wait(b_o + 8 * w, (nt - 1) & 1);
                tc_fence_after();
            }
            constexpr float kOut = KIND == KV_Q4 ? 65536.0f : 1.0f;
            const int64_t n = r.q0 + t;
            const bool whole = p.splits == 1;
            const float f = !whole ? kOut : sum == 0.0f ? 0.0f : kOut / sum;
            const int64_t at = ((n * p.heads + h) * p.splits + part);
            if (live) {
                if (!whole)
                    p.wj_ml[at] = make_float2(m, sum);
                else if (p.lse)
                    p.lse[n * p.heads + h] = lse_of(m, sum);
            }
            // out through the warp's own rows of Q's place (the products that read it have ended), so
            // that rows leave whole: fp16 results in one go, fp32 partial ones in halves
            const uint32_t mine = sq + w * TILE + (row & 96) * 128;
            auto unit_at = [&](int rw, int u) { return mine + (u >> 3) * 16384 + rw * 128 + (((u & 7) ^ (rw & 7)) << 4); };
            char *const own = !live  ? nullptr
                              : whole ? (char *)(p.out + n * p.os + (int64_t)h * D)
                                      : (char *)(p.wj_o + at * D);
            constexpr int UNITS = D / 8;  // 16-byte units of a row in that place
#pragma unroll
            for (int part2 = 0; part2 < 2; ++part2) {
                if (whole && part2) break;
                uint32_t o[32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    if (!whole && c / (D / 64) != part2) continue;
                    if (nt > 0) {
                        tmem_ld32(to + 32 * c, o);
                        tc_wait_ld();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(o[i + k]) * f;
                        if (whole)
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(
                                             unit_at(lane, 4 * c + i / 8) + 2 * (i & 4)),
                                         "r"(pack_h2(x[0], x[1])), "r"(pack_h2(x[2], x[3]))
                                         : "memory");
                        else
                            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             unit_at(lane, 8 * (c % (D / 64)) + i / 4)),
                                         "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3])
                                         : "memory");
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < UNITS; ++i) {
                    constexpr int RPI = 32 / UNITS;
                    const int rw = i * RPI + lane / UNITS, u = lane % UNITS;
                    char *d = reinterpret_cast<char *>(__shfl_sync(~0u, (unsigned long long)own, rw));
                    if (d) *reinterpret_cast<uint4 *>(d + part2 * 2 * D + 16 * u) = lds128(unit_at(rw, u));
                }
                __syncwarp();
            }
        }
    done:;
    } else {
        if constexpr (!QUANT) reg_shrink<C::REGS_LO>();
        if (warp == 8) {
            // ---- MMA
            if (nt > 0 && elect_one()) {
                if (two)
                    mma_thread<KIND, D, true>(tmem, sq, skv, b_full, b_empty, b_q, b_s, b_sf, b_p, b_o, nt, wait);
                else
                    mma_thread<KIND, D, false>(tmem, sq, skv, b_full, b_empty, b_q, b_s, b_sf, b_p, b_o, nt, wait);
                if (dead) {  // the products in flight end before tensor memory is freed
                    tc_commit(b_end);
                    mbar_wait(b_end, 0);
                }
            }
        } else if (!QUANT && (warp == 9 || warp == 10)) {
            // ---- fp16: warp 9 brings the K tiles, warp 10 the V tiles, record by record (pieces
            // of 16 tokens x 64 numbers = 2 KB by bulk copies); a V record that the context or the
            // window cuts is copied by hand with its stale rows zeroed, and V records outside are
            // zero.  The page numbers of the next tile are asked for while this one is copied
            // (each in its turn, by one warp: 3860 cycles a key tile instead of ~2400).
            const int which = warp - 9;
            const int vlo = p.window > 0 ? max(0, r.L - r.T - p.window + 1) : 0;
            const int64_t pages = p.kv.slots >> p.kv.page_shift;
            const int half = lane >> 3;  // lane = record + 8 half
            auto page_of = [&](int it) -> int {
                const int rec = 8 * (j0 + it) + (lane & 7);
                if (it >= nt || rec * 16 >= r.L || rec * 16 + 16 <= vlo) return 0;
                return p.table[b * p.table_stride + ((rec << 4) >> p.kv.page_shift)];
            };
            int next = page_of(0);
            for (int it = 0; it < nt; ++it) {
                const int i = which ? 2 * it + 2 : max(0, 2 * it - 1), jt = j0 + it;  // K0 K1 V0 K2 V1 ..
                const uint32_t dst = skv + (i % NS) * TILE, full = b_full + 8 * (i % NS);
                const int rec = 8 * jt + (lane & 7);
                const bool any = rec * 16 < r.L && rec * 16 + 16 > vlo;
                const bool cut = rec * 16 + 16 > r.L || rec * 16 < vlo;
                int64_t pg = next;
                next = page_of(it + 1);
                if (pg < 0 || pg >= pages) {
                    pg = 0;
                    atomicOr(p.err, kStatusRange);
                }
                const uint8_t *src = p.kv.pool +
                    (((pg * p.kv.heads + kh) << (p.kv.page_shift - 4)) +
                     (rec & ((1 << (p.kv.page_shift - 4)) - 1))) * kv_record_bytes(KV_F16, D) +
                    which * 32 * D;
                wait(b_empty + 8 * (i % NS), ((i / NS) & 1) ^ 1);
                const bool copy = !dead && half < C::HALVES && any && !(which && cut);
                if (copy) {
                    mbar_arrive_expect_tx(full, 2048);
                    bulk_g2s(dst + half * 16384 + (lane & 7) * 2048, src + half * 2048, 2048, full);
                }
                uint32_t by_hand = __ballot_sync(~0u, which && cut && lane < 8);
                while (by_hand) {
                    const int k = __ffs(by_hand) - 1;
                    by_hand &= by_hand - 1;
                    const uint8_t *s = reinterpret_cast<const uint8_t *>(
                        __shfl_sync(~0u, (unsigned long long)src, k));
                    const bool some = __shfl_sync(~0u, (int)any, k);
                    for (int x = lane; x < 2 * D; x += 32) {  // 16-byte units: half, token, unit
                        const int tok = (8 * jt + k) * 16 + (x >> 3) % 16;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (some && tok >= vlo && tok < r.L) v = *reinterpret_cast<const uint4 *>(s + 16 * x);
                        const uint32_t at = dst + (x >> 7) * 16384 + k * 2048 + (x & 127) * 16;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x),
                                     "r"(v.y), "r"(v.z), "r"(v.w)
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();  // all of the warp's stores before the last arrivals
                if (!copy) mbar_arrive(full);
            }
            if (__any_sync(~0u, dead))  // the copies in flight land before the CTA ends
                for (int it = max(0, nt - NS); it < nt; ++it) {
                    const int i = which ? 2 * it + 2 : max(0, 2 * it - 1);
                    mbar_wait(b_full + 8 * (i % NS), (i / NS) & 1);
                }
        } else if (QUANT && warp == 9) {
            // ---- codes: the K or V rows of a key tile's records as they are, one record a lane,
            // and with K the records' steps and multipliers
            const int vlo = p.window > 0 ? max(0, r.L - r.T - p.window + 1) : 0;
            const int64_t pages = p.kv.slots >> p.kv.page_shift;
            constexpr int ROWS = 16 * kv_row_bytes(KIND, D);
            if (lane < 8) {
                auto page_of = [&](int it) -> int {
                    const int rec = 8 * (j0 + it) + lane;
                    if (it >= nt || rec * 16 >= r.L || rec * 16 + 16 <= vlo) return -1;
                    const int pg = p.table[b * p.table_stride + ((rec << 4) >> p.kv.page_shift)];
                    if (pg >= 0 && pg < pages) return pg;
                    atomicOr(p.err, kStatusRange);
                    return 0;
                };
                auto src_of = [&](int it, int pg) {
                    const int rec = 8 * (j0 + it) + lane;
                    return p.kv.pool + ((((int64_t)pg * p.kv.heads + kh) << (p.kv.page_shift - 4)) +
                                        (rec & ((1 << (p.kv.page_shift - 4)) - 1))) * kv_record_bytes(KIND, D);
                };
                int page0 = -1, page1 = page_of(0), page2 = page_of(1);  // of key tiles it - 1, it, it + 1
                int slot = 0, phase = 0;
                auto copy = [&](int it, int pg, int which) {
                    wait(b_out + 8 * slot, phase ^ 1);
                    if (pg >= 0 && !dead) {
                        const uint8_t *src = src_of(it, pg);
                        mbar_arrive_expect_tx(b_in + 8 * slot, ROWS + (which ? 0 : C::SMALL));
                        bulk_g2s(stage + slot * C::PART + lane * ROWS, src + which * ROWS, ROWS, b_in + 8 * slot);
                        if (!which)
                            bulk_g2s(small + ((it & 3) * 8 + lane) * C::SMALL, src + 2 * ROWS, C::SMALL,
                                     b_in + 8 * slot);
                    } else {
                        mbar_arrive(b_in + 8 * slot);
                    }
                    if (++slot == C::PARTS) slot = 0, phase ^= 1;
                };
                for (int it = 0; it < nt; ++it) {  // K0 K1 V0 K2 V1 ..
                    copy(it, page1, 0);
                    if (it > 0) copy(it - 1, page0, 1);
                    page0 = page1, page1 = page2, page2 = page_of(it + 2);
                }
                if (nt > 0) copy(nt - 1, page0, 1);
                if (dead)  // the copies in flight land before the CTA ends
                    for (int i = 0; i < C::PARTS; ++i) mbar_wait(b_in + 8 * i, i < slot ? phase : phase ^ 1, kWaitLimit);
            }
        } else if (QUANT && warp >= 12) {
            // ---- codes: 128 threads decode them into the operand tiles.  Thread `tid` takes the
            // 16-byte unit stored at place `un` of row `tok` of every (128 / R)th record.
            constexpr int R = kv_row_bytes(KIND, D);  // also the units of a record's K (V) rows
            constexpr int UPR = R / 16;               // units of a row
            constexpr int STEP = 128 / R;             // records between a thread's units
            const int tid = threadIdx.x & 127;
            const int vlo = p.window > 0 ? max(0, r.L - r.T - p.window + 1) : 0;
            const int tok = tid % R / UPR, un = tid % UPR, rec0 = tid / R;
            const int u = (int)((kv_unit(KIND, D, tok, un) >> 4) % UPR);  // which unit of the row lies there
            const int mu_at = 128 + tok * (D / 32) + (KIND == KV_Q8 ? u >> 1 : u);
            const float ksc = fabsf(p.scale) * 1.4426950408889634f * (KIND == KV_Q4 ? 65536.0f : 1.0f);
            int sslot = 0, sphase = 0, slot = 0, phase = 0;
            auto decode = [&](int it, int which) {
                wait(b_in + 8 * sslot, sphase);
                wait(b_empty + 8 * slot, phase ^ 1);
                if (!which) {
                    // steps of the key tile's token tid
                    const int j = ((j0 + it) << 7) + tid;
                    const uint32_t st = small + ((it & 3) * 8 + (tid >> 4)) * C::SMALL + 4 * (tid & 15);
                    float ck = 0.0f, vs = 0.0f;
                    if (j >= vlo && j < r.L) ck = lds_f(st) * ksc, vs = lds_f(st + 64);
                    float *sc = scales + (it & 3) * 384;
                    sc[tid] = ck;
                    sc[128 + tid] = fmaxf(log2f(vs), -40.0f) + (vs - vs);  // (a NaN stays one)
                    sc[256 + tid] = 1.0f / fmaxf(vs, 0x1p-40f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_sc + 8 * (it & 3));
                }
                const uint32_t src = stage + sslot * C::PART + tid * 16, dst = skv + slot * TILE;
                const uint32_t sm = small + (it & 3) * 8 * C::SMALL + mu_at + which * 16 * (D / 32);
#pragma unroll
                for (int rec = 0; rec < 8; rec += STEP) {
                    const uint4 c = lds128(src + rec * R * 16);
                    const uint32_t mb = mult_byte<KIND>(lds8(sm + (rec + rec0) * C::SMALL)) & 255;
                    const uint32_t mm = mult_h2(mb, mb), f = mult_scale<KIND>(mm), sh = mult_shift<KIND>(mm);
                    const int row = (rec + rec0) * 16 + tok;
                    const uint32_t line = dst + row * 128;
                    auto put = [&](int d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {  // numbers d .. d + 7
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         line + (d >> 6) * 16384 + ((((d >> 3) & 7) ^ (row & 7)) << 4)),
                                     "r"(a0), "r"(a1), "r"(a2), "r"(a3)
                                     : "memory");
                    };
                    // (the order of a unit's stores depends on which half of the numbers it is in,
                    // so that eight lanes' stores never meet in a bank)
                    if constexpr (KIND == KV_Q8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int k = i ^ ((u >> 2) & 1);
                            const uint32_t y0 = (k ? c.z : c.x) ^ 0x80808080u, y1 = (k ? c.w : c.y) ^ 0x80808080u;
                            put(16 * u + 8 * k, hfma2(__byte_perm(y0, 0x64646464u, 0x4140), f, sh),
                                hfma2(__byte_perm(y0, 0x64646464u, 0x4342), f, sh),
                                hfma2(__byte_perm(y1, 0x64646464u, 0x4140), f, sh),
                                hfma2(__byte_perm(y1, 0x64646464u, 0x4342), f, sh));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // low nibbles of 8 bytes, twice, and the high ones
                            const int hi = (i >> 1) ^ ((u >> 1) & 1);
                            const uint32_t y0 = ((i & 1 ? c.z : c.x) >> (4 * hi)) & 0x0f0f0f0fu;
                            const uint32_t y1 = ((i & 1 ? c.w : c.y) >> (4 * hi)) & 0x0f0f0f0fu;
                            put(32 * u + 16 * hi + 8 * (i & 1), hfma2(__byte_perm(y0, 0, 0x4140), f, sh),
                                hfma2(__byte_perm(y0, 0, 0x4342), f, sh), hfma2(__byte_perm(y1, 0, 0x4140), f, sh),
                                hfma2(__byte_perm(y1, 0, 0x4342), f, sh));
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(b_full + 8 * slot);
                    mbar_arrive(b_out + 8 * sslot);
                }
                if (++sslot == C::PARTS) sslot = 0, sphase ^= 1;
                if (++slot == NS) slot = 0, phase ^= 1;
            };
            for (int it = 0; it < nt; ++it) {
                decode(it, 0);
                if (it > 0) decode(it - 1, 1);
            }
            if (++slot == NS) slot = 0, phase ^= 1;  // K(nt) does not exist
            if (nt > 0) decode(nt - 1, 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace qg
