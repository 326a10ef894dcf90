// The row-wise operators of the paged key / value cache:
//
// k_paged_write: projected rows to finished queries and cache pages in one
// pass.  Per head of hd dims:  y = x / sqrt(mean(x^2) + eps) * w (optional),
// the first R dims turned by the row's (cos, sin), then q -> 16 bits, k and
// v -> the pages' format.  An 8-bit head keeps one f32 scale s = max|y| / L
// (L = 127 or 448; 1 for a head of zeros) and codes of y / s.
//
// k_paged_read: pages to contiguous rows.
//
// Both are bound by HBM traffic (a dozen flops an element): every element is
// read once and written once.  A head of hd dims is the work of hd / 8 lanes,
// 8 dims each (k_paged_read: 16 codes each for 8-bit pages, 16-byte pieces),
// so the norm's sum and the largest magnitude are a few shuffles inside one
// warp.  A lane of k_paged_write holds both dims of each pair that the rotation
// turns: four from each half (or four neighbours and the next four), so the
// rotation needs none, at the price of 8-byte loads of 16-bit rows (full
// 32-byte sectors all the same).
//
// Measured: 13,500 rows of 28 + 2 x 4 heads of 128, bf16 into e4m3 pages with
// norms and rotation, 59.4 us (4.4 TB/s; the f32 arithmetic of the norm, the
// rotation and the codes takes the issue slots that are left over); 155,000
// positions of int8 read into bf16 100 us (5.9 TB/s, 87% of a plain copy's
// rate); 8 rows of a decode step 2.6 us, a launch and one load's latency.
#include <cuda_fp8.h>

#include "paged.cuh"
#include "paged.h"

namespace qwen2 {
namespace paged {

namespace {

constexpr int kRowThreads = 128;

// Four elements of a row, as they lie in memory and as f32.
template <int DT>
struct Raw4 {
    uint32_t w[DT == QWEN2_DTYPE_F32 ? 4 : 2];
};
template <int DT>
__device__ __forceinline__ Raw4<DT> load4(const char* p) {
    Raw4<DT> r;
    if constexpr (DT == QWEN2_DTYPE_F32) {
        const uint4 v = ld_stream_v4(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
        r.w[2] = v.z;
        r.w[3] = v.w;
    } else {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p));
    }
    return r;
}
template <int DT>
__device__ __forceinline__ void to_f32(const Raw4<DT>& r, float* x) {
#pragma unroll
    for (int j = 0; j < (DT == QWEN2_DTYPE_F32 ? 4 : 2); ++j) {
        if constexpr (DT == QWEN2_DTYPE_F32) {
            x[j] = __uint_as_float(r.w[j]);
        } else {
            float2 f;
            if constexpr (DT == QWEN2_DTYPE_F16) f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[j]));
            else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.w[j]));
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8_16(const float (&x)[8], bool bf16) {
    return make_uint4(pack2(x[0], x[1], bf16), pack2(x[2], x[3], bf16), pack2(x[4], x[5], bf16),
                      pack2(x[6], x[7], bf16));
}

__device__ __forceinline__ uint2 pack4_16(const float* x, bool bf16) {
    return make_uint2(pack2(x[0], x[1], bf16), pack2(x[2], x[3], bf16));
}

// max that keeps a NaN, so that a head holding one gets a NaN scale instead
// of losing it.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t int8_code(float y) {
    // Half away from zero, as the weights' Q8_0 blocks are rounded.
    return (uint32_t)(uint8_t)(int8_t)fminf(fmaxf(roundf(y), -127.f), 127.f);
}

// Four 8-bit codes of x / scale, the quotient taken as x times 1 / scale (a
// division an element was a third of the kernel's instructions).
template <int FMT>
__device__ __forceinline__ uint32_t pack4_8(const float* x, float inv) {
    const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
    if constexpr (FMT == QWEN2_KV_INT8)
        return int8_code(y[0]) | int8_code(y[1]) << 8 | int8_code(y[2]) << 16 | int8_code(y[3]) << 24;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// The sequence that holds `row`: the number of sequences that end at or before
// it.  Up to 256 sequences are counted by the warp's lanes, all loads in
// flight at once; more go by bisection.  `start` is ascending; if it is not,
// the result is still inside [0, n_seq].
__device__ __forceinline__ int find_seq(const int* start, int n_seq, int row, int lane) {
    if (n_seq <= 256) {
        int c = 0;
        for (int i = 1 + lane; i <= n_seq; i += 32) c += __ldg(start + i) <= row;
        return __reduce_add_sync(0xffffffffu, c);
    }
    int lo = 0, hi = n_seq;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(start + mid + 1) <= row) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

struct WriteArgs {
    Pool kv;
    Batch b;
    Rows q, q_out, k, v;
    const float *q_norm, *k_norm;
    const float* rope;
    float eps;
    int rope_rows, rotary, interleaved;
    int n_head;         // 0: no queries
    int slices;         // warps one row's heads are spread over
    int out_bf16;
};

// A pair turned by an angle's (cos, sin).
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
    const float t = fmaf(x, c, -__fmul_rn(y, s));
    y = fmaf(y, c, __fmul_rn(x, s));
    x = t;
}

template <int N>
struct Int {
    static constexpr int value = N;
};

// One warp per (row, slice of its heads): a row's lookups and rotation factors
// are loaded once and serve all its heads.
template <int DT, int FMT, int HD>
__global__ void __launch_bounds__(kRowThreads, 6) k_paged_write(const __grid_constant__ WriteArgs a) {
    constexpr int kLanes = HD / 8;            // lanes per head
    constexpr int kHeads = 32 / kLanes;       // heads per warp step
    constexpr int kIn = DT == QWEN2_DTYPE_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const long long row_l = w / a.slices;
    if (row_l >= a.b.n_rows) return;
    const int row = (int)row_l, slice = (int)(w - row_l * a.slices);
    const int s = find_seq(a.b.q_start, a.b.n_seq, row, lane);
    if (s >= a.b.n_seq) return;
    const Seq q = load_seq(a.b, a.kv.page_shift, s);
    if (q.bad_rows || q.bad_len) {
        if (lane == 0) raise_guard(a.b.guard, q.bad_rows ? kGuardShape : kGuardPosition);
        return;
    }
    const int i = row - q.q0;
    if (i < 0 || i >= q.n) return;            // not this sequence's: q_start is not ascending, or row < q_start[0]
    const int pos = q.kv - q.n + i;
    if (pos < 0 || (a.rotary && pos >= a.rope_rows)) {
        if (lane == 0) raise_guard(a.b.guard, kGuardPosition);
        return;
    }
    const int page = __ldg(a.b.pages + (long long)s * a.b.pages_stride + (pos >> a.kv.page_shift));
    if ((unsigned)page >= (unsigned)a.kv.n_pages) {
        if (lane == 0) raise_guard(a.b.guard, QWEN2_GUARD_PAGE);
        return;
    }
    const int off = pos & ((1 << a.kv.page_shift) - 1);
    const int c = lane % kLanes, sub = lane / kLanes;

    // This lane's dims: d0 .. d0 + 3 and d1 .. d1 + 3, and the rotation of its four
    // pairs: (x[e], x[4 + e]) or, interleaved, (x[2 e], x[2 e + 1]).
    const int half = a.rotary >> 1;
    const bool split = !a.interleaved && 4 * c < half;          // a lane of the turning dims, half layout
    const bool turns = a.interleaved ? 8 * c < a.rotary : split;
    const int d0 = split ? 4 * c : 8 * c;
    const int d1 = split ? half + 4 * c : d0 + 4;
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (turns) {
        const float4* t = reinterpret_cast<const float4*>(a.rope + (long long)pos * a.rotary + 8 * c);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float4 f = __ldg(t + p);
            cs[2 * p] = f.x;
            sn[2 * p] = f.y;
            cs[2 * p + 1] = f.z;
            sn[2 * p + 1] = f.w;
        }
    }
    const long long kv_row = (long long)page * a.kv.page_bytes + (long long)off * a.kv.token_bytes;
    // Heads [h0, h1) of the queries (kKind 0), keys (1) or values (2); every lane
    // of the warp takes every step of kHeads heads, kBatch steps' loads in flight.
    const auto heads = [&](auto kind, int h0, int h1) {
        constexpr int kKind = decltype(kind)::value;
        constexpr int kBatch = kKind == 0 ? 4 : 2;
        const Rows& src = kKind == 0 ? a.q : kKind == 1 ? a.k : a.v;
        const char* from = src.data + (long long)row * src.row_bytes;
        const float* nw = kKind == 0 ? a.q_norm : kKind == 1 ? a.k_norm : nullptr;
        float w[8];
        if (kKind != 2 && nw) {
            const float4 w0 = __ldg(reinterpret_cast<const float4*>(nw + d0));
            const float4 w1 = __ldg(reinterpret_cast<const float4*>(nw + d1));
            w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
            w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
        }
        for (; h0 < h1; h0 += kBatch * kHeads) {
            Raw4<DT> raw[kBatch][2];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int h = min(h0 + b * kHeads + sub, h1 - 1);    // past the last head: its values, not stored
                const char* p = from + (long long)h * src.head_bytes;
                raw[b][0] = load4<DT>(p + kIn * d0);
                raw[b][1] = load4<DT>(p + kIn * d1);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (h0 + b * kHeads >= h1) break;
                const int h = h0 + b * kHeads + sub;
                float x[8];
                to_f32<DT>(raw[b][0], x);
                to_f32<DT>(raw[b][1], x + 4);
                if (kKind != 2 && nw) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float r = rsqrtf(ss * (1.f / HD) + a.eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
                }
                if (kKind != 2 && a.rotary) {
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) turn(x[2 * e], x[2 * e + 1], cs[e], sn[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) turn(x[e], x[4 + e], cs[e], sn[e]);
                    }
                }
                if constexpr (kKind == 0) {
                    if (h < h1) {
                        char* dst = a.q_out.data + (long long)row * a.q_out.row_bytes + (long long)h * a.q_out.head_bytes;
                        *reinterpret_cast<uint2*>(dst + 2 * d0) = pack4_16(x, a.out_bf16);
                        *reinterpret_cast<uint2*>(dst + 2 * d1) = pack4_16(x + 4, a.out_bf16);
                    }
                } else {
                    char* dst = (kKind == 1 ? a.kv.k : a.kv.v) + kv_row + (long long)h * a.kv.head_bytes;
                    if constexpr (FMT == QWEN2_KV_F16 || FMT == QWEN2_KV_BF16) {
                        if (h < h1) {
                            *reinterpret_cast<uint2*>(dst + 2 * d0) = pack4_16(x, FMT == QWEN2_KV_BF16);
                            *reinterpret_cast<uint2*>(dst + 2 * d1) = pack4_16(x + 4, FMT == QWEN2_KV_BF16);
                        }
                    } else {
                        float m = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(x[e]));
#pragma unroll
                        for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const float scale = m == 0.f ? 1.f : __fdiv_rn(m, FMT == QWEN2_KV_INT8 ? 127.f : 448.f);
                        if (h < h1) {
                            const float inv = __fdiv_rn(1.f, scale);
                            *reinterpret_cast<uint32_t*>(dst + d0) = pack4_8<FMT>(x, inv);
                            *reinterpret_cast<uint32_t*>(dst + d1) = pack4_8<FMT>(x + 4, inv);
                            if (c == 0)
                                (kKind == 1 ? a.kv.k_scale
                                            : a.kv.v_scale)[(((long long)page * a.kv.n_kv + h) << a.kv.page_shift) + off] = scale;
                        }
                    }
                }
            }
        }
    };
    // This warp's share of the row's steps.
    const int sq = (a.n_head + kHeads - 1) / kHeads, sk = (a.kv.n_kv + kHeads - 1) / kHeads;
    const int s0 = (sq + 2 * sk) * slice / a.slices, s1 = (sq + 2 * sk) * (slice + 1) / a.slices;
    heads(Int<0>{}, kHeads * s0, min(a.n_head, kHeads * s1));
    heads(Int<1>{}, kHeads * max(0, s0 - sq), min(a.kv.n_kv, kHeads * (s1 - sq)));
    heads(Int<2>{}, kHeads * max(0, s0 - sq - sk), min(a.kv.n_kv, kHeads * (s1 - sq - sk)));
}

struct ReadArgs {
    Pool kv;
    Batch b;
    Rows k, v;
    const int* out_start;
    int n_out;
};

// Codes or 16-bit values as f32.
template <int FMT, int N>
__device__ __forceinline__ void widen(const uint4& raw, float (&x)[N]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (FMT == QWEN2_KV_F16 || FMT == QWEN2_KV_BF16) {
            float2 f;
            if constexpr (FMT == QWEN2_KV_F16) f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else if constexpr (FMT == QWEN2_KV_INT8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = (float)(int8_t)(w[i] >> (8 * j));
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                x[4 * i + 2 * j] = f.x;
                x[4 * i + 2 * j + 1] = f.y;
            }
        }
    }
}

// A warp takes kReadRows consecutive output rows: lane l looks up row l (one
// chain of dependent loads for all of them), then the warp streams their heads.
constexpr int kReadRows = 4;

template <int FMT, int DT, int HD>
__global__ void __launch_bounds__(kRowThreads) k_paged_read(const __grid_constant__ ReadArgs a) {
    constexpr bool k8 = FMT == QWEN2_KV_INT8 || FMT == QWEN2_KV_E4M3;
    constexpr int kN = k8 ? 16 : 8;           // dims per lane
    constexpr int kLanes = HD / kN;
    constexpr int kHeads = 32 / kLanes;
    constexpr int kOut = DT == QWEN2_DTYPE_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kReadRows;
    if (first >= a.n_out) return;
    int page = -1, off = 0;
    if (lane < kReadRows && first + lane < a.n_out) {
        const int row = (int)first + lane;
        int lo = 0, hi = a.b.n_seq;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.out_start + mid + 1) <= row) lo = mid + 1;
            else hi = mid;
        }
        if (lo < a.b.n_seq) {
            const int pos = row - __ldg(a.out_start + lo);
            const int kv = __ldg(a.b.kv_len + lo);
            const bool bad_len = kv < 0 || kv > ((long long)a.b.max_pages << a.kv.page_shift);
            if (bad_len) raise_guard(a.b.guard, kGuardPosition);
            else if (pos >= 0 && pos < kv) {
                page = __ldg(a.b.pages + (long long)lo * a.b.pages_stride + (pos >> a.kv.page_shift));
                off = pos & ((1 << a.kv.page_shift) - 1);
                if ((unsigned)page >= (unsigned)a.kv.n_pages) {
                    raise_guard(a.b.guard, QWEN2_GUARD_PAGE);
                    page = -1;
                }
            }
        }
    }
    const int c = lane % kLanes, sub = lane / kLanes;
    const int n_slots = 2 * a.kv.n_kv;
#pragma unroll
    for (int r = 0; r < kReadRows; ++r) {
        const int pg = __shfl_sync(0xffffffffu, page, r), of = __shfl_sync(0xffffffffu, off, r);
        if (pg < 0) continue;
        for (int slot = sub; slot < n_slots; slot += kHeads) {
            const bool is_v = slot >= a.kv.n_kv;
            const int h = is_v ? slot - a.kv.n_kv : slot;
            const char* src = (is_v ? a.kv.v : a.kv.k) + (long long)pg * a.kv.page_bytes +
                              (long long)of * a.kv.token_bytes + (long long)h * a.kv.head_bytes + 16 * c;
            const uint4 raw = ld_stream_v4(src);
            float x[kN];
            widen<FMT, kN>(raw, x);
            if constexpr (k8) {
                const float s = __ldg((is_v ? a.kv.v_scale : a.kv.k_scale) +
                                      (((long long)pg * a.kv.n_kv + h) << a.kv.page_shift) + of);
#pragma unroll
                for (int e = 0; e < kN; ++e) x[e] *= s;
            }
            const Rows& o = is_v ? a.v : a.k;
            char* dst = o.data + (first + r) * o.row_bytes + (long long)h * o.head_bytes + (long long)kN * kOut * c;
            if constexpr (DT == QWEN2_DTYPE_F32) {
#pragma unroll
                for (int e = 0; e < kN / 4; ++e)
                    reinterpret_cast<float4*>(dst)[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < kN / 8; ++e) {
                    const float y[8] = {x[8 * e], x[8 * e + 1], x[8 * e + 2], x[8 * e + 3],
                                        x[8 * e + 4], x[8 * e + 5], x[8 * e + 6], x[8 * e + 7]};
                    reinterpret_cast<uint4*>(dst)[e] = pack8_16(y, DT == QWEN2_DTYPE_BF16);
                }
            }
        }
    }
}

template <int DT, int FMT>
cudaError_t launch_write_hd(const WriteArgs& a, int head_dim, cudaStream_t st) {
    const long long warps = (long long)a.b.n_rows * a.slices;
    const unsigned blocks = (unsigned)((warps + kRowThreads / 32 - 1) / (kRowThreads / 32));
    if (head_dim == 64) k_paged_write<DT, FMT, 64><<<blocks, kRowThreads, 0, st>>>(a);
    else k_paged_write<DT, FMT, 128><<<blocks, kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_write_fmt(const WriteArgs& a, int format, int head_dim, cudaStream_t st) {
    switch (format) {
        case QWEN2_KV_F16: return launch_write_hd<DT, QWEN2_KV_F16>(a, head_dim, st);
        case QWEN2_KV_BF16: return launch_write_hd<DT, QWEN2_KV_BF16>(a, head_dim, st);
        case QWEN2_KV_INT8: return launch_write_hd<DT, QWEN2_KV_INT8>(a, head_dim, st);
        default: return launch_write_hd<DT, QWEN2_KV_E4M3>(a, head_dim, st);
    }
}

template <int FMT, int DT>
cudaError_t launch_read_hd(const ReadArgs& a, int head_dim, cudaStream_t st) {
    const int per = kRowThreads / 32 * kReadRows;
    const unsigned blocks = (unsigned)((a.n_out + (long long)per - 1) / per);
    if (head_dim == 64) k_paged_read<FMT, DT, 64><<<blocks, kRowThreads, 0, st>>>(a);
    else k_paged_read<FMT, DT, 128><<<blocks, kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_read_dt(const ReadArgs& a, int dtype, int head_dim, cudaStream_t st) {
    switch (dtype) {
        case QWEN2_DTYPE_F32: return launch_read_hd<FMT, QWEN2_DTYPE_F32>(a, head_dim, st);
        case QWEN2_DTYPE_F16: return launch_read_hd<FMT, QWEN2_DTYPE_F16>(a, head_dim, st);
        default: return launch_read_hd<FMT, QWEN2_DTYPE_BF16>(a, head_dim, st);
    }
}

}  // namespace

cudaError_t enqueue_write(const Pool& kv, const Batch& b, const qwen2_paged_write_opts* o, int format, int head_dim,
                          int n_head, int dtype, bool out_bf16, const Rows& q, const Rows& q_out, const Rows& k,
                          const Rows& v, cudaStream_t st) {
    WriteArgs a{};
    a.kv = kv;
    a.b = b;
    a.q = q;
    a.q_out = q_out;
    a.k = k;
    a.v = v;
    a.n_head = n_head;
    a.out_bf16 = out_bf16;
    if (o) {
        a.q_norm = n_head ? o->q_norm : nullptr;
        a.k_norm = o->k_norm;
        a.eps = o->norm_eps;
        a.rope = o->rope;
        a.rope_rows = o->rope_rows;
        a.rotary = o->rope ? o->rotary_dim : 0;
        a.interleaved = o->interleaved;
    }
    // One warp per row once the rows alone fill the device (12 warps an SM),
    // so that a row's lookups are made once; with fewer rows its heads are
    // spread over as many warps as do, down to one step of heads each (a decode
    // step's few rows are then one round of loads).  Five chunks of 200 to 700
    // rows of 28 + 2 x 4 heads of 128 into int8 take 18.8 us so, 21.3 us with 16
    // and 22.2 us with 48 warps an SM wanted.
    const int heads = head_dim == 64 ? 4 : 2;
    const int steps = (n_head + heads - 1) / heads + 2 * ((kv.n_kv + heads - 1) / heads);
    a.slices = (int)min((long long)steps, (152 * 12 + (long long)b.n_rows - 1) / b.n_rows);
    switch (dtype) {
        case QWEN2_DTYPE_F32: return launch_write_fmt<QWEN2_DTYPE_F32>(a, format, head_dim, st);
        case QWEN2_DTYPE_F16: return launch_write_fmt<QWEN2_DTYPE_F16>(a, format, head_dim, st);
        default: return launch_write_fmt<QWEN2_DTYPE_BF16>(a, format, head_dim, st);
    }
}

cudaError_t enqueue_read(const Pool& kv, const Batch& b, int format, int head_dim, const int* out_start, int n_out,
                         int dtype, const Rows& k, const Rows& v, cudaStream_t st) {
    ReadArgs a{kv, b, k, v, out_start, n_out};
    switch (format) {
        case QWEN2_KV_F16: return launch_read_dt<QWEN2_KV_F16>(a, dtype, head_dim, st);
        case QWEN2_KV_BF16: return launch_read_dt<QWEN2_KV_BF16>(a, dtype, head_dim, st);
        case QWEN2_KV_INT8: return launch_read_dt<QWEN2_KV_INT8>(a, dtype, head_dim, st);
        default: return launch_read_dt<QWEN2_KV_E4M3>(a, dtype, head_dim, st);
    }
}

}  // namespace paged
}  // namespace qwen2
