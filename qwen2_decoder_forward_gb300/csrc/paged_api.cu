// C entries of the paged key / value cache operators: argument checks (all
// of them before anything is launched) and the host-side rotation table.
#include <math.h>
#include <stdint.h>

#include <exception>
#include <new>
#include <string>

#include "ctx.h"
#include "paged.cuh"
#include "paged.h"

using namespace qwen2;
using namespace qwen2::paged;

namespace {

int refuse(int code, const std::string& msg) {
    set_thread_error(msg);
    return code;
}
// Who refuses what; put together only when a message needs it.
struct Where {
    const char *fn, *name;
    std::string operator+(const char* msg) const { return std::string(fn) + (name ? std::string(": ") + name : "") + msg; }
};

bool mult16(long long bytes) { return bytes >= 0 && bytes % 16 == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int dtype_size(int dt) { return dt == QWEN2_DTYPE_F32 ? 4 : 2; }

// Nothing a host-side check does may leave a C entry as an exception.
template <class F>
int guarded(const char* what, F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return QWEN2_E_OOM;
    } catch (...) {
        try {
            set_thread_error(std::string(what) + ": unexpected exception");
        } catch (...) {
        }
        return QWEN2_E_CUDA;
    }
}

constexpr long long kMaxStride = 1ll << 40;   // elements; keeps every offset inside 64 bits

int check_pool(const char* fn, const qwen2_paged_kv* c, Pool& p) {
    const Where at{fn, nullptr};
    if (!c) return refuse(QWEN2_E_ARG, at + ": kv is NULL");
    if (c->format < QWEN2_KV_F16 || c->format > QWEN2_KV_E4M3)
        return refuse(QWEN2_E_UNSUPPORTED, at + ": page format " + std::to_string(c->format) + " is not supported");
    if (c->head_dim != 64 && c->head_dim != 128)
        return refuse(QWEN2_E_UNSUPPORTED, at + ": head_dim " + std::to_string(c->head_dim) + " is not supported (64 or 128)");
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return refuse(QWEN2_E_UNSUPPORTED, at + ": page_size " + std::to_string(c->page_size) +
                                               " is not supported (16, 32, 64, 128 or 256)");
    if (c->n_pages < 1 || c->n_kv_head < 1 || c->n_kv_head > 1024)
        return refuse(QWEN2_E_ARG, at + ": n_pages and n_kv_head must be positive (at most 1024 kv heads)");
    if (!c->k || !c->v) return refuse(QWEN2_E_ARG, at + ": k or v is NULL");
    const bool k8 = c->format == QWEN2_KV_INT8 || c->format == QWEN2_KV_E4M3;
    const int size = k8 ? 1 : 2;
    for (long long s : {(long long)c->page_stride, (long long)c->token_stride, (long long)c->head_stride})
        if (s < 0 || s > kMaxStride || !mult16(s * size))
            return refuse(QWEN2_E_ARG, at + ": page strides must be non-negative multiples of 16 bytes");
    if (!aligned16(c->k) || !aligned16(c->v)) return refuse(QWEN2_E_ARG, at + ": k and v must be 16-byte aligned");
    if (k8 && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
        return refuse(QWEN2_E_ARG, at + ": 8-bit pages need 16-byte aligned k_scale and v_scale");
    p.k = static_cast<char*>(c->k);
    p.v = static_cast<char*>(c->v);
    p.k_scale = k8 ? c->k_scale : nullptr;
    p.v_scale = k8 ? c->v_scale : nullptr;
    p.n_pages = c->n_pages;
    p.page_shift = 4;
    while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
    p.n_kv = c->n_kv_head;
    p.page_bytes = c->page_stride * size;
    p.token_bytes = c->token_stride * size;
    p.head_bytes = c->head_stride * size;
    return QWEN2_OK;
}

int check_batch(const char* fn, const qwen2_paged_batch* c, int page_size, bool rows, Batch& b) {
    const Where at{fn, nullptr};
    if (!c) return refuse(QWEN2_E_ARG, at + ": batch is NULL");
    if (c->n_seq < 1 || c->n_seq > 4096) return refuse(QWEN2_E_ARG, at + ": n_seq outside [1, 4096]");
    if (!c->kv_len || !c->pages || (rows && !c->q_start)) return refuse(QWEN2_E_ARG, at + ": null batch array");
    if (rows && (c->n_rows < 0 || c->max_q < 0)) return refuse(QWEN2_E_ARG, at + ": n_rows and max_q must be >= 0");
    if (c->max_pages < 1 || c->pages_stride < c->max_pages)
        return refuse(QWEN2_E_ARG, at + ": max_pages must be >= 1 and pages_stride >= max_pages");
    if (c->pages_stride > kMaxStride) return refuse(QWEN2_E_ARG, at + ": pages_stride too large");
    if ((long long)c->max_pages * page_size > 1ll << 30)
        return refuse(QWEN2_E_UNSUPPORTED, at + ": more than 2^30 positions per sequence");
    b.n_seq = c->n_seq;
    b.n_rows = c->n_rows;
    b.max_q = c->max_q;
    b.max_pages = c->max_pages;
    b.pages_stride = c->pages_stride;
    b.q_start = c->q_start;
    b.kv_len = c->kv_len;
    b.pages = c->pages;
    b.guard = c->guard;
    return QWEN2_OK;
}

int check_rows(const char* fn, const char* name, const qwen2_rows* r, Rows& o) {
    const Where at{fn, name};
    if (!r || !r->data) return refuse(QWEN2_E_ARG, at + " is NULL");
    if (r->dtype < QWEN2_DTYPE_F32 || r->dtype > QWEN2_DTYPE_BF16)
        return refuse(QWEN2_E_UNSUPPORTED, at + " has an unknown dtype");
    const int size = dtype_size(r->dtype);
    for (long long s : {(long long)r->row_stride, (long long)r->head_stride})
        if (s < 0 || s > kMaxStride || !mult16(s * size))
            return refuse(QWEN2_E_ARG, at + ": strides must be non-negative multiples of 16 bytes");
    if (!aligned16(r->data)) return refuse(QWEN2_E_ARG, at + " must be 16-byte aligned");
    o.data = static_cast<char*>(r->data);
    o.row_bytes = r->row_stride * size;
    o.head_bytes = r->head_stride * size;
    return QWEN2_OK;
}

int check_heads(const char* fn, int n_head, int n_kv, int n_rows) {
    if (n_head < 1 || n_head % n_kv)
        return refuse(QWEN2_E_ARG, std::string(fn) + ": n_head must be a positive multiple of n_kv_head");
    if (n_head / n_kv > 64) return refuse(QWEN2_E_UNSUPPORTED, std::string(fn) + ": more than 64 query heads per kv head");
    if ((long long)n_rows * n_head >= 1ll << 31)
        return refuse(QWEN2_E_UNSUPPORTED, std::string(fn) + ": n_rows * n_head must be below 2^31");
    return QWEN2_OK;
}

int launched(const char* fn, cudaError_t e) {
    if (e == cudaSuccess) return QWEN2_OK;
    return refuse(QWEN2_E_CUDA, std::string(fn) + ": launch failed: " + cudaGetErrorString(e));
}

// SMs of the current device (looked up once per device).
int sm_count(int* out) {
    static int known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return refuse(QWEN2_E_CUDA, "no usable current CUDA device");
    }
    int n = dev < 64 ? __atomic_load_n(&known[dev], __ATOMIC_RELAXED) : 0;
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return refuse(QWEN2_E_CUDA, "cannot read the SM count");
        }
        if (dev < 64) __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
    }
    *out = n;
    return QWEN2_OK;
}

}  // namespace

extern "C" {

int qwen2_rope_table(int32_t rows, int32_t rotary_dim, double theta, const qwen2_rope_scaling* s, float* table) {
    return guarded("qwen2_rope_table", [&]() -> int {
        const char* fn = "qwen2_rope_table: ";
        if (!table || rows < 1 || rotary_dim < 2 || rotary_dim % 2 || !(theta > 0.0) || !std::isfinite(theta))
            return refuse(QWEN2_E_ARG, std::string(fn) + "table NULL, rows < 1, rotary_dim odd or theta not positive");
        const int kind = s ? s->kind : QWEN2_ROPE_PLAIN;
        if (kind < QWEN2_ROPE_PLAIN || kind > QWEN2_ROPE_YARN)
            return refuse(QWEN2_E_UNSUPPORTED, std::string(fn) + "unknown scaling kind");
        const double factor = kind == QWEN2_ROPE_PLAIN ? 1.0 : s->factor;
        if (!(factor >= 1.0) || !std::isfinite(factor)) return refuse(QWEN2_E_ARG, std::string(fn) + "factor must be >= 1");
        const int half = rotary_dim / 2;
        double lo = 0, hi = 0, gain = 1;
        if (kind == QWEN2_ROPE_YARN) {
            if (s->original_rows < 1 || !(s->beta_slow > 0.0) || !(s->beta_fast > s->beta_slow) || !(theta > 1.0) ||
                !std::isfinite(s->beta_fast))
                return refuse(QWEN2_E_ARG, std::string(fn) + "YARN needs original_rows >= 1, beta_fast > beta_slow > 0, theta > 1");
            // The dim whose angle turns `beta` times within original_rows positions.
            const auto dim = [&](double beta) {
                return rotary_dim * log(s->original_rows / (beta * 2.0 * 3.14159265358979323846)) / (2.0 * log(theta));
            };
            lo = fmax(floor(dim(s->beta_fast)), 0.0);
            hi = fmin(ceil(dim(s->beta_slow)), (double)rotary_dim - 1);
            if (hi <= lo) hi = lo + 0.001;
            gain = factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
        }
        for (int i = 0; i < half; ++i) {
            double inv = pow(theta, -2.0 * i / rotary_dim);
            if (kind == QWEN2_ROPE_LINEAR) inv /= factor;
            if (kind == QWEN2_ROPE_YARN) {
                const double slow = fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);   // 1: divided by factor
                inv = inv * (1.0 - slow) + inv / factor * slow;
            }
            for (int p = 0; p < rows; ++p) {
                const double a = (double)p * inv;
                table[((int64_t)p * half + i) * 2] = (float)(cos(a) * gain);
                table[((int64_t)p * half + i) * 2 + 1] = (float)(sin(a) * gain);
            }
        }
        return QWEN2_OK;
    });
}

int qwen2_paged_write(const qwen2_paged_kv* kv, const qwen2_paged_batch* batch, const qwen2_paged_write_opts* opts,
                      int32_t n_head, const qwen2_rows* q, const qwen2_rows* q_out, const qwen2_rows* k,
                      const qwen2_rows* v, void* stream) {
    return guarded("qwen2_paged_write", [&]() -> int {
        const char* fn = "qwen2_paged_write";
        Pool p{};
        Batch b{};
        Rows rq{}, ro{}, rk{}, rv{};
        int r = check_pool(fn, kv, p);
        if (r == QWEN2_OK) r = check_batch(fn, batch, kv->page_size, true, b);
        if (r == QWEN2_OK) r = check_rows(fn, "k", k, rk);
        if (r == QWEN2_OK) r = check_rows(fn, "v", v, rv);
        if (r != QWEN2_OK) return r;
        if (!q != !q_out) return refuse(QWEN2_E_ARG, "qwen2_paged_write: q and q_out go together");
        if (q) {
            r = check_rows(fn, "q", q, rq);
            if (r == QWEN2_OK) r = check_rows(fn, "q_out", q_out, ro);
            if (r == QWEN2_OK) r = check_heads(fn, n_head, kv->n_kv_head, b.n_rows);
            if (r != QWEN2_OK) return r;
            if (q_out->dtype == QWEN2_DTYPE_F32)
                return refuse(QWEN2_E_UNSUPPORTED, "qwen2_paged_write: q_out must be f16 or bf16");
        }
        if (k->dtype != v->dtype || (q && q->dtype != k->dtype))
            return refuse(QWEN2_E_ARG, "qwen2_paged_write: q, k and v must have one dtype");
        if (opts) {
            if (opts->rope) {
                if (opts->rotary_dim < 16 || opts->rotary_dim > kv->head_dim || opts->rotary_dim % 16)
                    return refuse(QWEN2_E_UNSUPPORTED,
                                  "qwen2_paged_write: rotary_dim must be a multiple of 16, at most head_dim");
                if (opts->rope_rows < 1) return refuse(QWEN2_E_ARG, "qwen2_paged_write: rope_rows must be >= 1");
                if (!aligned16(opts->rope)) return refuse(QWEN2_E_ARG, "qwen2_paged_write: rope must be 16-byte aligned");
            }
            if ((opts->q_norm && !aligned16(opts->q_norm)) || (opts->k_norm && !aligned16(opts->k_norm)))
                return refuse(QWEN2_E_ARG, "qwen2_paged_write: q_norm and k_norm must be 16-byte aligned");
            if ((opts->q_norm || opts->k_norm) && !(opts->norm_eps >= 0.f))
                return refuse(QWEN2_E_ARG, "qwen2_paged_write: norm_eps must be >= 0");
        }
        if (b.n_rows == 0) return QWEN2_OK;
        return launched(fn, enqueue_write(p, b, opts, kv->format, kv->head_dim, q ? n_head : 0, k->dtype,
                                          q && q_out->dtype == QWEN2_DTYPE_BF16, rq, ro, rk, rv,
                                          static_cast<cudaStream_t>(stream)));
    });
}

int qwen2_paged_read(const qwen2_paged_kv* kv, const qwen2_paged_batch* batch, const int32_t* out_start, int32_t n_out,
                     const qwen2_rows* k, const qwen2_rows* v, void* stream) {
    return guarded("qwen2_paged_read", [&]() -> int {
        const char* fn = "qwen2_paged_read";
        Pool p{};
        Batch b{};
        Rows rk{}, rv{};
        int r = check_pool(fn, kv, p);
        if (r == QWEN2_OK) r = check_batch(fn, batch, kv->page_size, false, b);
        if (r == QWEN2_OK) r = check_rows(fn, "k", k, rk);
        if (r == QWEN2_OK) r = check_rows(fn, "v", v, rv);
        if (r != QWEN2_OK) return r;
        if (!out_start || n_out < 0) return refuse(QWEN2_E_ARG, "qwen2_paged_read: out_start NULL or n_out < 0");
        if (k->dtype != v->dtype) return refuse(QWEN2_E_ARG, "qwen2_paged_read: k and v must have one dtype");
        if (n_out == 0) return QWEN2_OK;
        return launched(fn, enqueue_read(p, b, kv->format, kv->head_dim, out_start, n_out, k->dtype, rk, rv,
                                         static_cast<cudaStream_t>(stream)));
    });
}

int64_t qwen2_paged_attention_workspace(const qwen2_paged_kv* kv, const qwen2_paged_batch* batch, int32_t n_head) {
    int64_t bytes = -1;
    guarded("qwen2_paged_attention_workspace", [&]() -> int {
        const char* fn = "qwen2_paged_attention_workspace";
        Pool p{};
        Batch b{};
        int n_sm = 0;
        int r = check_pool(fn, kv, p);
        if (r == QWEN2_OK) r = check_batch(fn, batch, kv->page_size, true, b);
        if (r == QWEN2_OK) r = check_heads(fn, n_head, kv->n_kv_head, b.n_rows);
        if (r == QWEN2_OK) r = sm_count(&n_sm);
        if (r == QWEN2_OK) bytes = attn_workspace(b, p, kv->head_dim, n_head, n_sm);
        return r;
    });
    return bytes;
}

int qwen2_paged_attention(const qwen2_paged_kv* kv, const qwen2_paged_batch* batch, int32_t n_head,
                          const qwen2_rows* q, const qwen2_rows* out, float* lse, float scale, int32_t causal,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    return guarded("qwen2_paged_attention", [&]() -> int {
        const char* fn = "qwen2_paged_attention";
        Pool p{};
        Batch b{};
        Rows rq{}, ro{};
        int r = check_pool(fn, kv, p);
        if (r == QWEN2_OK) r = check_batch(fn, batch, kv->page_size, true, b);
        if (r == QWEN2_OK) r = check_heads(fn, n_head, kv->n_kv_head, b.n_rows);
        if (r == QWEN2_OK) r = check_rows(fn, "q", q, rq);
        if (r == QWEN2_OK) r = check_rows(fn, "out", out, ro);
        if (r != QWEN2_OK) return r;
        if (q->dtype == QWEN2_DTYPE_F32 || out->dtype != q->dtype)
            return refuse(QWEN2_E_UNSUPPORTED, "qwen2_paged_attention: q must be f16 or bf16, and out the same");
        if ((kv->format == QWEN2_KV_F16 && q->dtype != QWEN2_DTYPE_F16) ||
            (kv->format == QWEN2_KV_BF16 && q->dtype != QWEN2_DTYPE_BF16))
            return refuse(QWEN2_E_UNSUPPORTED, "qwen2_paged_attention: 16-bit pages need queries of their own type");
        if (!std::isfinite(scale)) return refuse(QWEN2_E_ARG, "qwen2_paged_attention: scale must be finite");
        if (b.n_rows == 0) return QWEN2_OK;
        int n_sm = 0;
        if ((r = sm_count(&n_sm)) != QWEN2_OK) return r;
        const int64_t need = attn_workspace(b, p, kv->head_dim, n_head, n_sm);
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need)
            return refuse(QWEN2_E_ARG, "qwen2_paged_attention: workspace must be 256-byte aligned and of at least " +
                                           std::to_string(need) + " bytes");
        AttnCall c{kv->format, kv->head_dim, n_head, q->dtype, causal != 0, scale, lse, workspace};
        return launched(fn, enqueue_attention(p, b, c, rq, ro, n_sm, static_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
