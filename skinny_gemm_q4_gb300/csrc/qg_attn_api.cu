// C ABI of the attention side: cache, rotation and attention handles, argument
// checks and launches.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <vector>

#include "qg_attn_launch.cuh"
#include "qgemv.h"

using namespace qg;

namespace qg {
void set_last_error(const char *msg);  // qg_api.cu: the text qgemv_last_error returns
cudaError_t read_error_word(unsigned int *word, uint32_t *w, bool clear);  // qg_api.cu
}

struct qg_kv {
    int kind;
    int64_t pages;
    int page_size, page_shift, heads, dim, device, sms;
    uint8_t *pool;
    unsigned int *err;
};

struct qg_rope {
    qg_rope_desc d;
    float mscale;
    int device, sms;
    uint64_t *freq;  // rot_dim / 2 fractions of a turn
};

struct qg_attn {
    qg_attn_desc d;
    int device, sms;
    unsigned int *err;
    float *ws_o;    // partial results of contexts cut into leaves (null: one leaf at most)
    float2 *ws_ml;
    float *wj_o;    // partial results of keys cut into parts (null: they never are)
    float2 *wj_ml;
};

namespace {

qg_status fail(qg_status s, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

qg_status cuda_fail(cudaError_t e, const char *what)
{
    return fail(QG_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// After a launch: its own error, and with QGEMV_DEBUG_SYNC the asynchronous ones.
qg_status launched(cudaError_t e, const char *what, cudaStream_t s)
{
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e, what);
    }
    const char *v = getenv("QGEMV_DEBUG_SYNC");
    if (v && *v && strcmp(v, "0") != 0) {
        e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return cuda_fail(e, what);
    }
    return QG_OK;
}

// A zeroed device word.
qg_status new_word(unsigned int **w)
{
    *w = nullptr;
    cudaError_t e = cudaMalloc((void **)w, sizeof(unsigned int));
    if (e == cudaSuccess) e = cudaMemset(*w, 0, sizeof(unsigned int));
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // (streams that do not wait for the null one)
    if (e == cudaSuccess) return QG_OK;
    cudaGetLastError();
    if (*w) cudaFree(*w);
    *w = nullptr;
    return fail(QG_ENOMEM, "error word allocation failed (%s)", cudaGetErrorName(e));
}

qg_status read_word(unsigned int *w, uint32_t *flags_out, int clear)
{
    const cudaError_t e = read_error_word(w, flags_out, clear != 0);
    return e == cudaSuccess ? QG_OK : cuda_fail(e, "error word");
}

int log2_of(int v)
{
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

bool dim_ok(int d) { return d == 64 || d == 128; }

// Most new tokens of a request that the decode kernel takes.
int few_tokens(const qg_attn_desc &d, int max_q)
{
    return std::max(1, std::min(max_q, kDecRows / (d.q_heads / d.kv_heads)));
}

// A handle's memory is on the device that it was made on: its launches go there only, and two
// handles of a call are of one device.
qg_status check_current(int device)
{
    int now = 0;
    const cudaError_t e = cudaGetDevice(&now);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    if (now != device)
        return fail(QG_EINVAL, "the handle was made on device %d, and device %d is current", device, now);
    return QG_OK;
}

qg_status check_cache_device(const qg_kv *c, int device)
{
    if (c->device == device) return QG_OK;
    return fail(QG_EINVAL, "the cache was made on device %d, the handle on device %d", c->device, device);
}

// One [N][heads][dim] fp16 argument: pointer (none for no tokens), alignment, token stride (0
// becomes contiguous).
qg_status check_heads(const char *name, const void *p, int64_t *stride, int heads, int dim,
                      int64_t N)
{
    if (!p && N > 0) return fail(QG_EINVAL, "null %s", name);
    if (!aligned(p, 16)) return fail(QG_EALIGN, "%s is not 16-byte aligned", name);
    const int64_t least = (int64_t)heads * dim;
    if (*stride == 0) *stride = least;
    if (*stride < least && N > 1)
        return fail(QG_EINVAL, "%s: token stride %lld below %lld", name, (long long)*stride,
                    (long long)least);
    if (*stride % 8) return fail(QG_EALIGN, "%s: token stride is not a multiple of 8", name);
    return QG_OK;
}

qg_status check_count(int64_t N)
{
    if (N < 0 || N > 0x7fffffff) return fail(QG_EINVAL, "N = %lld tokens", (long long)N);
    return QG_OK;
}

KvView view_of(const qg_kv *c)
{
    KvView v;
    v.pool = c->pool;
    v.slots = c->pages * c->page_size;
    v.page_shift = c->page_shift;
    v.heads = c->heads;
    v.err = c->err;
    return v;
}

qg_status freqs_of(const qg_rope_desc *d, double *f, double *mscale)
{
    if (!d || !f || !mscale) return fail(QG_EINVAL, "null argument");
    if (!dim_ok(d->head_dim)) return fail(QG_EUNSUPPORTED, "head_dim %d", d->head_dim);
    if (d->rot_dim < 16 || d->rot_dim > d->head_dim || d->rot_dim % 16)
        return fail(QG_EUNSUPPORTED, "rot_dim %d: a multiple of 16 up to head_dim", d->rot_dim);
    if (d->layout != QG_ROPE_HALF && d->layout != QG_ROPE_INTERLEAVED)
        return fail(QG_EINVAL, "layout %d", d->layout);
    if (d->scaling < QG_ROPE_SCALE_NONE || d->scaling > QG_ROPE_SCALE_BANDS)
        return fail(QG_EINVAL, "scaling %d", d->scaling);
    if (!(d->base > 1.0) || !std::isfinite(d->base)) return fail(QG_EINVAL, "base %g", d->base);
    const bool scaled = d->scaling != QG_ROPE_SCALE_NONE;
    if (scaled && (!(d->factor >= 1.0) || !std::isfinite(d->factor)))
        return fail(QG_EINVAL, "factor %g", d->factor);
    const bool by_turns = d->scaling == QG_ROPE_SCALE_YARN || d->scaling == QG_ROPE_SCALE_BANDS;
    const double low = d->low != 0.0 ? d->low : 1.0;
    const double high =
        d->high != 0.0 ? d->high : d->scaling == QG_ROPE_SCALE_YARN ? 32.0 : 4.0;
    if (by_turns && (!(d->original_len > 0.0) || !std::isfinite(d->original_len) ||
                     !(low > 0.0) || !(high > low) || !std::isfinite(high)))
        return fail(QG_EINVAL, "original_len %g, low %g, high %g", d->original_len, low, high);
    if (!(d->mscale >= 0.0) || !std::isfinite(d->mscale))
        return fail(QG_EINVAL, "mscale %g", d->mscale);
    const int half = d->rot_dim / 2;
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < half; ++i) {
        const double f0 = pow(d->base, -2.0 * i / d->rot_dim);
        if (d->scaling == QG_ROPE_SCALE_LINEAR) {
            f[i] = f0 / d->factor;
        } else if (d->scaling == QG_ROPE_SCALE_YARN) {
            // the pair index that turns n times in original_len
            auto at = [&](double n) {
                return d->rot_dim * log(d->original_len / (n * two_pi)) / (2.0 * log(d->base));
            };
            const double lo = fmax(0.0, floor(at(high))),
                         hi = fmin((double)d->rot_dim - 1.0, ceil(at(low)));
            const double r = fmin(1.0, fmax(0.0, (i - lo) / fmax(hi - lo, 0.001)));
            f[i] = f0 / d->factor * r + f0 * (1.0 - r);
        } else if (d->scaling == QG_ROPE_SCALE_BANDS) {
            const double keep =
                fmin(1.0, fmax(0.0, (d->original_len * f0 / two_pi - low) / (high - low)));
            f[i] = f0 * keep + f0 / d->factor * (1.0 - keep);
        } else {
            f[i] = f0;
        }
    }
    *mscale = d->mscale != 0.0                          ? d->mscale
              : d->scaling == QG_ROPE_SCALE_YARN ? 0.1 * log(d->factor) + 1.0
                                                        : 1.0;
    return QG_OK;
}

}  // namespace

extern "C" {

int64_t qgemv_kv_page_bytes(qg_kv_type t, int32_t page_size, int32_t kv_heads, int32_t head_dim)
{
    if ((int)t < KV_F16 || (int)t > KV_Q4 || !dim_ok(head_dim)) return -1;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return -1;
    if (kv_heads < 1 || kv_heads > 1024) return -1;
    return (int64_t)kv_heads * (page_size / 16) * kv_record_bytes((int)t, head_dim);
}

qg_status qgemv_kv_create(qg_kv **out, qg_kv_type t, int64_t pages, int32_t page_size,
                          int32_t kv_heads, int32_t head_dim, void *pool_dev)
{
    if (!out) return fail(QG_EINVAL, "null output handle pointer");
    *out = nullptr;
    if (qgemv_kv_page_bytes(t, page_size, kv_heads, head_dim) < 0)
        return fail(QG_EUNSUPPORTED, "cache type %d, page_size %d, kv_heads %d, head_dim %d",
                    (int)t, page_size, kv_heads, head_dim);
    if (pages < 1 || pages > 0x7fffffff) return fail(QG_EINVAL, "%lld pages", (long long)pages);
    if (!pool_dev) return fail(QG_EINVAL, "null pool");
    if (!aligned(pool_dev, 16)) return fail(QG_EALIGN, "pool is not 16-byte aligned");
    qg_kv *c = new (std::nothrow) qg_kv();
    if (!c) return fail(QG_ENOMEM, "host allocation failed");
    c->kind = (int)t;
    c->pages = pages;
    c->page_size = page_size;
    c->page_shift = log2_of(page_size);
    c->heads = kv_heads;
    c->dim = head_dim;
    c->pool = (uint8_t *)pool_dev;
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&c->sms, cudaDevAttrMultiProcessorCount, c->device);
    qg_status st = e == cudaSuccess ? new_word(&c->err) : cuda_fail(e, "device query");
    if (st != QG_OK) {
        delete c;
        return st;
    }
    *out = c;
    return QG_OK;
}

qg_status qgemv_kv_write(qg_kv *c, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, const int64_t *slots, int64_t N, void *stream)
{
    if (!c || (!slots && N > 0)) return fail(QG_EINVAL, "null %s", c ? "slots" : "cache");
    qg_status st = check_count(N);
    if (st == QG_OK) st = check_heads("k", k, &k_stride, c->heads, c->dim, N);
    if (st == QG_OK) st = check_heads("v", v, &v_stride, c->heads, c->dim, N);
    if (st != QG_OK) return st;
    if (!aligned(slots, 8)) return fail(QG_EALIGN, "slots is not 8-byte aligned");
    if (N == 0) return QG_OK;
    st = check_current(c->device);
    if (st != QG_OK) return st;
    RopeParams p = {};
    p.k = (const __half *)k;
    p.v = (const __half *)v;
    p.ks = k_stride;
    p.vs = v_stride;
    p.slots = slots;
    p.nk = p.nv = c->heads;
    p.kv = view_of(c);
    return launched(launch_rope(p, c->kind, c->dim, true, N, c->sms, (cudaStream_t)stream),
                    "qgemv_kv_write", (cudaStream_t)stream);
}

qg_status qgemv_kv_read(qg_kv *c, const int64_t *slots, int64_t N, void *k_out, int64_t k_stride,
                        void *v_out, int64_t v_stride, void *stream)
{
    if (!c || (!slots && N > 0)) return fail(QG_EINVAL, "null %s", c ? "slots" : "cache");
    qg_status st = check_count(N);
    if (st == QG_OK) st = check_heads("k_out", k_out, &k_stride, c->heads, c->dim, N);
    if (st == QG_OK) st = check_heads("v_out", v_out, &v_stride, c->heads, c->dim, N);
    if (st != QG_OK) return st;
    if (!aligned(slots, 8)) return fail(QG_EALIGN, "slots is not 8-byte aligned");
    if (N == 0) return QG_OK;
    st = check_current(c->device);
    if (st != QG_OK) return st;
    KvReadParams p = {};
    p.kv = view_of(c);
    p.slots = slots;
    p.k = (__half *)k_out;
    p.v = (__half *)v_out;
    p.ks = k_stride;
    p.vs = v_stride;
    return launched(launch_kv_read(p, c->kind, c->dim, N, c->sms, (cudaStream_t)stream), "qgemv_kv_read",
                    (cudaStream_t)stream);
}

qg_status qgemv_kv_status(qg_kv *c, uint32_t *flags_out, int clear)
{
    if (!c || !flags_out) return fail(QG_EINVAL, "null argument");
    return read_word(c->err, flags_out, clear);
}

void qgemv_kv_destroy(qg_kv *c)
{
    if (!c) return;
    cudaFree(c->err);
    delete c;
}

qg_status qgemv_rope_freqs(const qg_rope_desc *d, double *freqs, double *mscale)
{
    return freqs_of(d, freqs, mscale);
}

qg_status qgemv_rope_create(qg_rope **out, const qg_rope_desc *d)
{
    if (!out) return fail(QG_EINVAL, "null output handle pointer");
    *out = nullptr;
    double f[64], ms;
    qg_status st = freqs_of(d, f, &ms);
    if (st != QG_OK) return st;
    // radians -> turns, as a fraction of 2^64; f is at most 1 radian
    uint64_t turns[64] = {};
    const int half = d->rot_dim / 2;
    for (int i = 0; i < half; ++i)
        turns[i] = (uint64_t)ldexpl((long double)f[i] / 6.283185307179586476925286766559L, 64);
    qg_rope *r = new (std::nothrow) qg_rope();
    if (!r) return fail(QG_ENOMEM, "host allocation failed");
    r->d = *d;
    r->mscale = (float)ms;
    cudaError_t e = cudaGetDevice(&r->device);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&r->sms, cudaDevAttrMultiProcessorCount, r->device);
    if (e == cudaSuccess) e = cudaMalloc((void **)&r->freq, sizeof turns);
    if (e != cudaSuccess) {
        cudaGetLastError();
        delete r;
        return fail(QG_ENOMEM, "frequency table: %s", cudaGetErrorName(e));
    }
    e = cudaMemcpy(r->freq, turns, sizeof turns, cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        cudaFree(r->freq);
        delete r;
        return cuda_fail(e, "frequency table");
    }
    *out = r;
    return QG_OK;
}

qg_status qgemv_rope_run(qg_rope *r, const qg_rope_args *a, void *stream)
{
    if (!r || !a) return fail(QG_EINVAL, "null %s", r ? "arguments" : "rotation");
    const int D = r->d.head_dim;
    qg_status st = check_count(a->N);
    if (st != QG_OK) return st;
    if (a->q_heads < 1 || a->q_heads > 65535 || a->kv_heads < 0 || a->kv_heads > 65535)
        return fail(QG_EINVAL, "%d q heads, %d kv heads", a->q_heads, a->kv_heads);
    RopeParams p = {};
    p.qs = a->q_stride, p.qos = a->q_out_stride;
    p.ks = a->k_stride, p.kos = a->k_out_stride, p.vs = a->v_stride;
    st = check_heads("q", a->q, &p.qs, a->q_heads, D, a->N);
    if (st == QG_OK) st = check_heads("q_out", a->q_out, &p.qos, a->q_heads, D, a->N);
    if (st == QG_OK && a->kv_heads) st = check_heads("k", a->k, &p.ks, a->kv_heads, D, a->N);
    if (st == QG_OK && a->kv_heads && (a->k_out || !a->cache))
        st = check_heads("k_out", a->k_out, &p.kos, a->kv_heads, D, a->N);
    if (st != QG_OK) return st;
    if (!a->positions && a->N > 0) return fail(QG_EINVAL, "null positions");
    if (!aligned(a->positions, 4)) return fail(QG_EALIGN, "positions is not 4-byte aligned");
    if ((a->q_weight || (a->k_weight && a->kv_heads)) && !(a->eps > 0.0f && std::isfinite(a->eps)))
        return fail(QG_EINVAL, "eps %g", (double)a->eps);
    if (!aligned(a->q_weight, 16) || !aligned(a->k_weight, 16))
        return fail(QG_EALIGN, "a norm weight is not 16-byte aligned");
    int kind = KV_NONE;
    if (a->cache) {
        const qg_kv *c = a->cache;
        if (c->dim != D || c->heads != a->kv_heads)
            return fail(QG_EINVAL, "the cache has %d heads of %d", c->heads, c->dim);
        st = check_cache_device(c, r->device);
        if (st != QG_OK) return st;
        if (!a->slots && a->N > 0) return fail(QG_EINVAL, "null slots");
        if (!aligned(a->slots, 8)) return fail(QG_EALIGN, "slots is not 8-byte aligned");
        st = check_heads("v", a->v, &p.vs, a->kv_heads, D, a->N);
        if (st != QG_OK) return st;
        kind = c->kind;
        p.kv = view_of(c);
        p.slots = a->slots;
        p.v = (const __half *)a->v;
        p.nv = a->kv_heads;
    }
    if (a->N == 0) return QG_OK;
    st = check_current(r->device);
    if (st != QG_OK) return st;
    p.q = (const __half *)a->q;
    p.k = (const __half *)a->k;
    p.qo = (__half *)a->q_out;
    p.ko = (__half *)a->k_out;
    p.qw = a->q_weight;
    p.kw = a->k_weight;
    p.eps = a->eps;
    p.mscale = r->mscale;
    p.pos = a->positions;
    p.freq = r->freq;
    p.nq = a->q_heads;
    p.nk = a->kv_heads;
    p.rot = r->d.rot_dim;
    return launched(launch_rope(p, kind, D, r->d.layout == QG_ROPE_HALF, a->N, r->sms,
                                (cudaStream_t)stream),
                    "qgemv_rope_run", (cudaStream_t)stream);
}

void qgemv_rope_destroy(qg_rope *r)
{
    if (!r) return;
    cudaFree(r->freq);
    delete r;
}

qg_status qgemv_attn_create(qg_attn **out, const qg_attn_desc *d)
{
    if (!out) return fail(QG_EINVAL, "null output handle pointer");
    *out = nullptr;
    if (!d) return fail(QG_EINVAL, "null description");
    if (!dim_ok(d->head_dim)) return fail(QG_EUNSUPPORTED, "head_dim %d", d->head_dim);
    if (d->kv_heads < 1 || d->kv_heads > 1024 || d->q_heads < 1 || d->q_heads % d->kv_heads)
        return fail(QG_EINVAL, "%d q heads, %d kv heads", d->q_heads, d->kv_heads);
    if (d->q_heads / d->kv_heads > 32)
        return fail(QG_EUNSUPPORTED, "%d q heads share a kv head", d->q_heads / d->kv_heads);
    if (d->max_tokens < 1 || d->max_tokens > (1 << 24) || d->max_batch < 1 ||
        d->max_batch > 65535 || d->max_len < 1 || d->max_len > (1 << 30))
        return fail(QG_EINVAL, "max_tokens %d, max_batch %d, max_len %lld", d->max_tokens,
                    d->max_batch, (long long)d->max_len);
    if ((int64_t)attn_leaves(d->max_len) * 2 * d->kv_heads > 0x7fffffff)
        return fail(QG_EUNSUPPORTED, "max_len %lld with %d kv heads", (long long)d->max_len,
                    d->kv_heads);
    qg_attn *a = new (std::nothrow) qg_attn();
    if (!a) return fail(QG_ENOMEM, "host allocation failed");
    a->d = *d;
    cudaError_t e = cudaGetDevice(&a->device);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&a->sms, cudaDevAttrMultiProcessorCount, a->device);
    qg_status st = e == cudaSuccess ? new_word(&a->err) : cuda_fail(e, "device query");
    if (st != QG_OK) {
        delete a;
        return st;
    }
    if (attn_leaves(d->max_len) > 1) {
        const int few_q = few_tokens(*d, d->max_tokens);
        const size_t tokens = std::min((size_t)d->max_batch * few_q, (size_t)d->max_tokens);
        const size_t rows = tokens * d->q_heads * attn_leaves(d->max_len);
        e = cudaMalloc((void **)&a->ws_o, rows * d->head_dim * sizeof(float));
        if (e == cudaSuccess) e = cudaMalloc((void **)&a->ws_ml, rows * sizeof(float2));
        if (e != cudaSuccess) {
            cudaGetLastError();
            qgemv_attn_destroy(a);
            return fail(QG_ENOMEM, "attention workspace of %zu rows failed", rows);
        }
    }
    if ((int64_t)d->max_tokens * (d->q_heads / d->kv_heads) > kDecRows && d->max_len >= 512) {
        // keys are cut (into parts of 256 at least) only while the CTAs, of at most 256 rows each,
        // do not fill the GPU
        const size_t rows = (size_t)256 * a->sms;
        e = cudaMalloc((void **)&a->wj_o, rows * d->head_dim * sizeof(float));
        if (e == cudaSuccess) e = cudaMalloc((void **)&a->wj_ml, rows * sizeof(float2));
        if (e != cudaSuccess) {
            cudaGetLastError();
            qgemv_attn_destroy(a);
            return fail(QG_ENOMEM, "attention workspace of %zu rows failed", rows);
        }
    }
    *out = a;
    return QG_OK;
}

qg_status qgemv_attn_run(qg_attn *h, const qg_attn_args *a, void *stream)
{
    if (!h || !a) return fail(QG_EINVAL, "null %s", h ? "arguments" : "attention handle");
    const qg_attn_desc &d = h->d;
    const qg_kv *c = a->cache;
    if (!c) return fail(QG_EINVAL, "null cache");
    if (c->dim != d.head_dim || c->heads != d.kv_heads)
        return fail(QG_EINVAL, "the cache has %d heads of %d", c->heads, c->dim);
    qg_status st = check_cache_device(c, h->device);
    if (st != QG_OK) return st;
    if (a->N < 0 || a->N > d.max_tokens || a->B < 1 || a->B > d.max_batch)
        return fail(QG_EINVAL, "N = %lld of at most %d tokens, B = %d of at most %d requests",
                    (long long)a->N, d.max_tokens, a->B, d.max_batch);
    if (a->max_q < (a->N > 0) || a->max_q > d.max_tokens)
        return fail(QG_EINVAL, "max_q = %d", a->max_q);
    if (a->causal != 0 && a->causal != 1) return fail(QG_EINVAL, "causal = %d", a->causal);
    if (a->window < 0) return fail(QG_EINVAL, "window = %d", a->window);
    if (!std::isfinite(a->scale)) return fail(QG_EINVAL, "scale is not finite");
    int64_t qs = a->q_stride, os = a->out_stride;
    st = check_heads("q", a->q, &qs, d.q_heads, d.head_dim, a->N);
    if (st == QG_OK) st = check_heads("out", a->out, &os, d.q_heads, d.head_dim, a->N);
    if (st != QG_OK) return st;
    if (!a->q_start || !a->kv_len || !a->page_table)
        return fail(QG_EINVAL, "null q_start, kv_len or page_table");
    if (!aligned(a->q_start, 4) || !aligned(a->kv_len, 4) || !aligned(a->page_table, 4) ||
        !aligned(a->lse, 4))
        return fail(QG_EALIGN, "q_start, kv_len, page_table or lse is not 4-byte aligned");
    if (a->table_width < 0 || (a->table_stride != 0 && a->table_stride < a->table_width))
        return fail(QG_EINVAL, "page table: width %d, stride %lld", a->table_width,
                    (long long)a->table_stride);
    if (a->N == 0) return QG_OK;
    st = check_current(h->device);
    if (st != QG_OK) return st;
    AttnParams p = {};
    p.kv = view_of(c);
    p.q = (const __half *)a->q;
    p.out = (__half *)a->out;
    p.lse = a->lse;
    p.qs = qs;
    p.os = os;
    p.q_start = a->q_start;
    p.kv_len = a->kv_len;
    p.table = a->page_table;
    p.table_stride = a->table_stride ? a->table_stride : a->table_width;
    p.N = a->N;
    p.B = a->B;
    p.max_q = a->max_q;
    p.heads = d.q_heads;
    p.group = d.q_heads / d.kv_heads;
    p.group_inv = 65536 / p.group + 1;
    // the longest context that the handle and the table allow
    p.max_len = (int)std::min(d.max_len, (int64_t)a->table_width * c->page_size);
    p.scale = a->scale;
    p.causal = a->causal;
    // A window of max_len positions hides nothing: a call without one.  (What is left is at most
    // 2^30 wide, so that the kernels' L - T - window fits 32 bits.)
    p.window = a->window >= p.max_len ? 0 : a->window;
    p.err = h->err;
    p.ws_o = h->ws_o;
    p.ws_ml = h->ws_ml;
    p.few_q = few_tokens(d, a->max_q);
    p.few_leaves = attn_leaves(p.max_len);
    const bool by_token = a->N < (int64_t)a->B * p.few_q;
    p.row_q = by_token;
    p.row_b = by_token ? 0 : p.few_q;
    p.row_parts = (p.few_q * p.group + 15) / 16;
    // Requests of few rows and the others go to different kernels; the host knows the sizes
    // when there is one request, or when all are of max_q tokens.
    const bool any_many = (a->B == 1 ? a->N : a->max_q) * p.group > kDecRows;
    const bool any_few = a->B == 1 ? !any_many : !any_many || a->N < (int64_t)a->B * a->max_q;
    // (a padded call's requests may be of few rows all the same: without the decode kernel the
    // chunk kernel takes every request)
    p.few_max = any_few ? kDecRows : 0;
    cudaError_t e = cudaSuccess;
    p.splits = 1;
    if (any_few) e = launch_attn_decode(p, c->kind, c->dim, h->sms, (cudaStream_t)stream);
    if (e == cudaSuccess && any_many) {
        p.wj_o = h->wj_o;
        p.wj_ml = h->wj_ml;
        // tile pairs of the requests, and the parts that their keys are cut into: as many as
        // still run at once, of two key tiles at least (128 tokens after 32768 in Q8: 90 us in 9
        // parts, 589 in one)
        const int per = 2 * (128 / p.group);
        const int64_t pairs = a->N == (int64_t)a->B * a->max_q
                                  ? (int64_t)a->B * ((a->max_q + per - 1) / per)
                                  : a->B + a->N / per;
        const int64_t room = h->sms / (pairs * d.kv_heads);
        p.splits = (int)std::max((int64_t)1, std::min(room, (int64_t)p.max_len / 256));
        e = launch_attn_chunk(p, c->kind, c->dim, pairs, (cudaStream_t)stream);
    }
    return launched(e, "qgemv_attn_run", (cudaStream_t)stream);
}

qg_status qgemv_attn_status(qg_attn *h, uint32_t *flags_out, int clear)
{
    if (!h || !flags_out) return fail(QG_EINVAL, "null argument");
    return read_word(h->err, flags_out, clear);
}

void qgemv_attn_destroy(qg_attn *h)
{
    if (!h) return;
    cudaFree(h->ws_o);
    cudaFree(h->ws_ml);
    cudaFree(h->wj_o);
    cudaFree(h->wj_ml);
    cudaFree(h->err);
    delete h;
}

}  // extern "C"
