// Attention over the paged cache for few new rows per sequence (single
// tokens, speculated tokens, short chunks), and the join of partial tiles.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = 2^(s_ij - m_i),
//   s_ij = scale log2(e) q_i . k_j,      m_i = max_j s_ij,
//
// taken in one pass over the keys with the running maximum and sum of each
// row (online softmax).  Bound by HBM: every cached byte is read once, for
// group * rows products of 2 hd flops, far below the tensor cores' rate.
//
// Split (paged.cuh): a tile is up to 8, 16 or 32 packed rows of one kv head,
// a unit 64 positions.  Inside a CTA warp w takes positions 16 w .. 16 w + 15
// of every unit on its own: its loads, softmax statistics and accumulators
// are the warp's, so the main loop has no block barrier.  The four warps meet
// at a tile's end in shared memory.  16 positions never cross a page, so a
// step needs one page lookup, loaded a step before its copies are issued (the
// first steps' all at once, a lane each).
//
// Loads: cp.async in 16-byte pieces, kStages steps in flight per warp, and
// positions past the tile's keys are filled with zeros instead of read (what
// a page holds there may be NaN).  Products: mma m16n8k16.  16 or 32 rows
// stand in M, positions (scores) or dims (values) in N.  Up to 8 rows, the
// single token of 8 or fewer query heads a kv head, stand in N, positions or
// dims in M: half the products, half the softmax and half the accumulators of
// a 16-row tile half empty, and the probabilities only need an 8 x 8
// transpose on their way into the second product.
//
// Measured (16 tokens over 8,000 - 32,700 positions of int8, 28 heads on 4,
// 346 MB): 73 us, 4.7 TB/s.  Instructions bound it, about 580 a step of 16
// positions and warp (a third of them widens the codes), which fill 64% of the
// issue slots with four CTAs an SM.  With the rows in M it took 88 us with
// three CTAs an SM and 115 us with two (the registers of 64 accumulators more,
// and a ring of four stages).  One token over 999 positions takes 8 us, of
// which the join and the two launches' latencies are some 4; the rest is a
// chain of a few load latencies (lengths, page ids, pages) per CTA, and so it
// is for 32 tokens over 256 - 4,095 of f16: 16.3 us for 36 MB.
//
// 8-bit pages: codes become exact f16 in registers (int8: 1024 + (c + 128)
// by a byte permute, minus 1152; e4m3: the hardware conversion) and the f32
// scales stay out of the products: the scores are multiplied by k's scale,
// the probabilities by v's, relative to G, the warp's largest v scale so far
// rounded up to a power of two, which the accumulators carry like the running
// maximum (f16 would lose small scales otherwise).  bf16 queries over 8-bit
// pages enter as f16 scaled by a power of two of their row's largest
// magnitude, which the scores are multiplied back by: exact but for dims
// below 2^-24 of the row's largest.
#include <cuda_fp8.h>

#include "paged.cuh"
#include "paged.h"

namespace qwen2 {
namespace paged {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 64;      // positions per unit
constexpr int kStep = 16;      // positions per warp and unit
constexpr int kCost = 1;       // slots of a tile beside its units (paged.cuh)

enum Kind { kSame16, kInt8, kE4m3 };

template <int HD, Kind K>
struct Shape {
    static constexpr int kSize = K == kSame16 ? 2 : 1;
    static constexpr int kRowBytes = HD * kSize;                   // one position of one head
    static constexpr int kTile = kStep * kRowBytes;                // K or V of a step
    static constexpr int kScales = K == kSame16 ? 0 : 2 * kStep * 4;
    static constexpr int kStage = 2 * kTile + kScales;
    static constexpr int kStages = kTile <= 1024 ? 6 : 3;
    static constexpr int kRing = kStage * kStages;                 // per warp
};

// Row tiles come in three forms: MT = 1 or 2 keeps 16 MT rows in the products'
// M (scores rows x positions), MT = 0 keeps 8 rows in N (scores positions x
// rows): half the products and half the softmax of a 16-row tile.
template <int MT>
constexpr int rows_of = MT ? 16 * MT : 8;
// CTAs an SM that the registers are held down to.
template <int MT>
constexpr int ctas_of = MT == 0 ? 4 : MT == 1 ? 3 : 2;

template <int HD, int MT>
struct Meet {   // where the warps meet
    // Two n tiles' 16 dims stand as 4 dims a lane of a quad (MT > 0), or the dims
    // g and g + 8 of an m tile side by side (MT = 0); the padding puts the rows
    // of one access into different banks.
    float o[rows_of<MT>][HD + (MT ? 16 : 4)];
    float m[kWarps][rows_of<MT>], l[kWarps][rows_of<MT>];
};

// 16-byte piece c of position r stands at piece c ^ f(r) of its row, so that
// both 8 rows' pieces of one column (ldmatrix) and 4 pieces of two adjacent
// rows (8-bit K) fall into all banks.
template <int RB>
__device__ __forceinline__ int swz(int r, int c) {
    if constexpr (RB == 64) return c ^ ((r >> 1) & 3);
    else return c ^ (((r & 1) << 2) | ((r >> 1) & 3));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Two codes of `w`, bytes (0,1) or (2,3) for FIRST = 0 / 2 and STEP = 1, bytes
// (0,2) or (1,3) for FIRST = 0 / 1 and STEP = 2, as exact f16.
template <Kind K, int FIRST, int STEP>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
    if constexpr (K == kInt8) {
        constexpr int sel = 0x4040 | FIRST | (FIRST + STEP) << 8;
        const uint32_t h = __byte_perm(w ^ 0x80808080u, 0x64646464u, sel);
        const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        constexpr int sel = 0x4400 | FIRST | (FIRST + STEP) << 4;
        const uint32_t p = STEP == 1 && FIRST == 0 ? w : __byte_perm(w, 0, sel);
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)p, __NV_E4M3);
        return (uint32_t)h.x | (uint32_t)h.y << 16;
    }
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Over the lanes of equal lane % 4.
__device__ __forceinline__ float col_max(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float col_sum(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The power of two at or above v, as an exponent in [-100, 100].
__device__ __forceinline__ int ceil_log2(float v) {
    const int b = __float_as_int(v);
    const int e = ((b >> 23) & 255) - 127 + ((b & 0x7fffff) != 0);
    return min(max(e, -100), 100);
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The copies of one warp step: cursor over the CTA's units, `ahead` steps
// before the products.
struct Feed {
    Tile t;
    int i;                 // unit within the tile's part
};

template <int HD, Kind K, bool BF16, int MT>
__global__ void __launch_bounds__(kThreads, ctas_of<MT>) k_paged_attn(const __grid_constant__ AttnArgs a) {
    using S = Shape<HD, K>;
    constexpr bool k8 = K != kSame16;
    constexpr bool kMmaBf16 = BF16 && !k8;
    constexpr bool kCols = MT == 0;              // rows in N
    constexpr int kRows = rows_of<MT>, kM = kCols ? 1 : MT, kH = kCols ? 1 : 2;
    constexpr int RB = S::kRowBytes;
    extern __shared__ __align__(128) unsigned char smem[];
    Meet<HD, MT>& meet = *reinterpret_cast<Meet<HD, MT>*>(smem);
    unsigned char* rings = smem + (sizeof(Meet<HD, MT>) + 127) / 128 * 128;
    long long* prefix = reinterpret_cast<long long*>(rings + kWarps * S::kRing);

    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const WorkList work = build_work<kUnit, kCost, kCost + 1>(a, prefix);
    bool open = false;
    if (work.begin < work.end) {
        const uint32_t ring = (uint32_t)__cvta_generic_to_shared(rings + warp * S::kRing);
        Tile t = find_tile<kUnit, kCost>(a, work);
        Feed f{t, 0};
        int f_page = -1;
        // Page of a step of the feed's tile; -1 if it has no keys, -2 if its id is bad.
        auto look_up = [&](int i) -> int {
            if (i >= f.t.n) return -1;
            const int key0 = (f.t.u0 + i) * kUnit + warp * kStep;
            if (key0 >= f.t.keys) return -1;
            const int p = __ldg(a.b.pages + (long long)f.t.s * a.b.pages_stride + (key0 >> a.kv.page_shift));
            return (unsigned)p < (unsigned)a.kv.n_pages ? p : -2;
        };
        unsigned bad = 0;     // per ring stage: its page id was bad
        // A lane copies piece lane % (RB / 16) of every kRowsAtOnce'th position.
        constexpr int kRowsAtOnce = 512 / RB;
        const long long lane_src = (long long)(lane / (RB / 16)) * a.kv.token_bytes + 16 * (lane % (RB / 16));
        const long long row_step = kRowsAtOnce * a.kv.token_bytes;
        // Issues the copies of the feed's step into `stage` and moves it on.
        auto issue = [&](int stage) {
            bad &= ~(1u << stage);
            if (f_page >= 0) {
                const int key0 = (f.t.u0 + f.i) * kUnit + warp * kStep;
                const int off = key0 & ((1 << a.kv.page_shift) - 1);
                const int n = f.t.keys - key0;       // positions of the step that are keys
                const long long at = (long long)f_page * a.kv.page_bytes + (long long)off * a.kv.token_bytes +
                                     (long long)f.t.head * a.kv.head_bytes;
                const uint32_t dst = ring + stage * S::kStage;
                // Positions past n are not read, though their page's memory is there.
                const char* ks = a.kv.k + at + lane_src;
                const char* vs = a.kv.v + at + lane_src;
#pragma unroll
                for (int i = 0; i < RB / 32; ++i) {
                    const int r = lane / (RB / 16) + i * kRowsAtOnce;
                    const uint32_t d = dst + r * RB + 16 * swz<RB>(r, lane % (RB / 16));
                    cp16(d, ks, r < n);
                    cp16(d + S::kTile, vs, r < n);
                    ks += row_step;
                    vs += row_step;
                }
                if constexpr (k8) {
                    if (lane < 8) {
                        const int c = lane & 3;
                        const float* sc = (lane < 4 ? a.kv.k_scale : a.kv.v_scale) +
                                          (((long long)f_page * a.kv.n_kv + f.t.head) << a.kv.page_shift) + off;
                        cp16(dst + 2 * S::kTile + 16 * lane, sc + 4 * c, true);
                    }
                }
            } else if (f_page == -2) {
                bad |= 1u << stage;
                if (lane == 0) raise_guard(a.b.guard, QWEN2_GUARD_PAGE);
            }
            cp_commit();
            if (f.t.n > 0 && ++f.i == f.t.n) {
                f.i = 0;
                next_tile<kUnit, kCost>(a, work, f.t);
            }
        };
        // The pages of the first steps come in one load, a lane each.
        const int first_pages = look_up(lane);
        const int first_n = t.n;
        bool begun = false;
        int stage = 0;

        for (;;) {
            // ---- a tile's part: queries ------------------------------------------
            const int packed0 = t.t * kRows, packed = t.q.n * a.group;
            uint32_t qf[kM][HD / 16][4];
            float rs[kM][2];           // factor of a row's scores
            int lim[kM][2];            // last position a row sees
            uint4 w[kM][kH][k8 ? HD / 32 : 1];
#pragma unroll
            for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                for (int h = 0; h < kH; ++h) {
                    const int i = packed0 + 16 * mt + 8 * h + g;
                    const bool in = i < packed;
                    const int row = t.q.q0 + (in ? i / a.group : 0), qh = t.head * a.group + (in ? i % a.group : 0);
                    const char* src = a.q.data + (long long)row * a.q.row_bytes + (long long)qh * a.q.head_bytes;
                    lim[mt][h] = in ? row_limit(a, t.q, i) : 0x7fffffff;
                    rs[mt][h] = a.scale_log2;
                    if constexpr (!k8) {
#pragma unroll
                        for (int k = 0; k < HD / 16; ++k) {
                            qf[mt][k][h] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 32 * k + 4 * t4)) : 0u;
                            qf[mt][k][2 + h] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + 32 * k + 16 + 4 * t4)) : 0u;
                        }
                    } else {
                        // Dims in the order the codes are read in: 4 codes of a word
                        // make the two halves of a k step's pairs.
#pragma unroll
                        for (int b = 0; b < HD / 64; ++b)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                w[mt][h][2 * b + j] =
                                    in ? __ldg(reinterpret_cast<const uint4*>(src + 128 * b + 32 * t4 + 16 * j))
                                       : make_uint4(0, 0, 0, 0);
                    }
                }
            // The first copies go out while the first queries come in.
            if (!begun) {
                begun = true;
#pragma unroll 1
                for (int st = 0; st < S::kStages - 1; ++st) {
                    f_page = st < first_n ? __shfl_sync(0xffffffffu, first_pages, st) : look_up(f.i);
                    issue(st);
                }
                f_page = look_up(f.i);
            }
            if constexpr (k8) {
#pragma unroll
                for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                    for (int h = 0; h < kH; ++h) {
                        uint4(&w1)[HD / 32] = w[mt][h];
                        if constexpr (BF16) {
                            float big = 0.f;
                            float x[HD / 4];
#pragma unroll
                            for (int j = 0; j < HD / 32; ++j) {
                                const uint32_t u[4] = {w1[j].x, w1[j].y, w1[j].z, w1[j].w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    x[8 * j + 2 * e] = __uint_as_float(u[e] << 16);
                                    x[8 * j + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
                                    big = fmaxf(big, fmaxf(fabsf(x[8 * j + 2 * e]), fabsf(x[8 * j + 2 * e + 1])));
                                }
                            }
                            const int e2 = ceil_log2(quad_max(big));
                            const float down = pow2i(-e2);
                            rs[mt][h] *= pow2i(e2);
#pragma unroll
                            for (int j = 0; j < HD / 32; ++j)
                                w1[j] = make_uint4(pack2<false>(x[8 * j] * down, x[8 * j + 1] * down),
                                                   pack2<false>(x[8 * j + 2] * down, x[8 * j + 3] * down),
                                                   pack2<false>(x[8 * j + 4] * down, x[8 * j + 5] * down),
                                                   pack2<false>(x[8 * j + 6] * down, x[8 * j + 7] * down));
                        }
#pragma unroll
                        for (int j = 0; j < HD / 32; ++j) {
                            qf[mt][2 * j][h] = w1[j].x;
                            qf[mt][2 * j][2 + h] = w1[j].y;
                            qf[mt][2 * j + 1][h] = w1[j].z;
                            qf[mt][2 * j + 1][2 + h] = w1[j].w;
                        }
                    }
            }
            if constexpr (kCols) {
                // The lane's scores are of rows 2 t4 and 2 t4 + 1.
                const float r = rs[0][0];
                const int last = lim[0][0];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    rs[0][j] = __shfl_sync(0xffffffffu, r, 8 * t4 + 4 * j);
                    lim[0][j] = __shfl_sync(0xffffffffu, last, 8 * t4 + 4 * j);
                }
            }
            const bool upper = packed - packed0 > kRows - 8;   // the last 8 rows hold any
            const int sure = row_limit(a, t.q, packed0);   // every row of the tile sees positions up to here
            constexpr int kTiles = kCols ? HD / 16 : HD / 8;
            float o[kM][kTiles][4];
            float m[kM][2], l[kM][2];
            int ge = -100;             // exponent of G
#pragma unroll
            for (int mt = 0; mt < kM; ++mt) {
#pragma unroll
                for (int d = 0; d < kTiles; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][d][e] = 0.f;
                m[mt][0] = m[mt][1] = -INFINITY;
                l[mt][0] = l[mt][1] = 0.f;
            }
            // ---- its units --------------------------------------------------------
            for (int i = 0; i < t.n; ++i) {
                cp_wait<S::kStages - 2>();
                __syncwarp();
                // The stage that the step before this one emptied is filled again.
                issue(stage == 0 ? S::kStages - 1 : stage - 1);
                f_page = look_up(f.i);
                const int key0 = (t.u0 + i) * kUnit + warp * kStep;
                const uint32_t kt = ring + stage * S::kStage, vt = kt + S::kTile;
                const bool skip = key0 >= t.keys || (bad >> stage & 1);
                if constexpr (kCols) {
                    if (!skip) {
                        const bool cut = key0 + kStep - 1 > sure || key0 + kStep > t.keys;
                        // scores: positions g and g + 8 of rows 2 t4 and 2 t4 + 1, in two chains
                        float c[2][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[0][e] = c[1][e] = 0.f;
                        const int r = (lane & 7) + ((lane >> 3) & 1) * 8, hi = lane >> 4;
                        if constexpr (!k8) {
#pragma unroll
                            for (int k = 0; k < HD / 16; ++k) {
                                uint32_t b[4];
                                ldsm4(kt + r * RB + 16 * swz<RB>(r, 2 * k + hi), b);
                                mma16816<kMmaBf16>(c[k & 1], b, qf[0][k][0], qf[0][k][2]);
                            }
                        } else {
#pragma unroll
                            for (int b = 0; b < HD / 64; ++b) {
                                uint32_t x[2][4];
#pragma unroll
                                for (int n = 0; n < 2; ++n)
                                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                                 : "=r"(x[n][0]), "=r"(x[n][1]), "=r"(x[n][2]), "=r"(x[n][3])
                                                 : "r"(kt + (8 * n + g) * RB + 16 * swz<RB>(8 * n + g, 4 * b + t4))
                                                 : "memory");
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t f[4] = {codes2<K, 0, 1>(x[0][k]), codes2<K, 0, 1>(x[1][k]),
                                                           codes2<K, 2, 1>(x[0][k]), codes2<K, 2, 1>(x[1][k])};
                                    mma16816<false>(c[k & 1], f, qf[0][4 * b + k][0], qf[0][4 * b + k][2]);
                                }
                            }
                        }
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = (c[0][e] + c[1][e]) * rs[0][e & 1];
                        float vs[2];
                        if constexpr (k8) {
                            float ks[2], top = 0.f;
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                const uint32_t sa = kt + 2 * S::kTile + 4 * (8 * n + g);
                                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks[n]) : "r"(sa) : "memory");
                                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs[n]) : "r"(sa + 64) : "memory");
                                // Positions that are no keys: whatever stands in the pool there is left out.
                                if (key0 + 8 * n + g >= t.keys) vs[n] = 0.f;
                                top = fmaxf(top, vs[n]);
                                v[2 * n] *= ks[n];
                                v[2 * n + 1] *= ks[n];
                            }
                            // A larger scale than G (the lane's own copy) moves it, in the whole warp.
                            if (__any_sync(0xffffffffu, ceil_log2(top) > ge)) {
                                const int ne = max(ge, ceil_log2(col_max(top)));
                                const float down = pow2i(max(ge - ne, -126));
#pragma unroll
                                for (int d = 0; d < kTiles; ++d)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[0][d][e] *= down;
                                ge = ne;
                            }
                            const float inv = pow2i(-ge);
                            vs[0] *= inv;
                            vs[1] *= inv;
                        }
                        if (cut) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (key0 + 8 * (e >> 1) + g > min(lim[0][e & 1], t.keys - 1)) v[e] = -INFINITY;
                        }
                        float corr[2];
                        bool moved = false;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float mn = fmaxf(m[0][j], col_max(fmaxf(v[j], v[2 + j])));
                            const float base = mn == -INFINITY ? 0.f : mn;
                            moved |= mn != m[0][j];
                            corr[j] = ex2(m[0][j] - base);
                            m[0][j] = mn;
                            v[j] = ex2(v[j] - base);
                            v[2 + j] = ex2(v[2 + j] - base);
                            l[0][j] = fmaf(l[0][j], corr[j], v[j] + v[2 + j]);
                        }
                        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                            for (int d = 0; d < kTiles; ++d)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[0][d][e] *= corr[e & 1];
                        }
                        if constexpr (k8) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] *= vs[e >> 1];
                        }
                        const uint32_t p0 = transpose8(pack2<kMmaBf16>(v[0], v[1]));
                        const uint32_t p1 = transpose8(pack2<kMmaBf16>(v[2], v[3]));
                        // values: dims in M, so that the rows stay in N
#pragma unroll
                        for (int d = 0; d < RB / 32; ++d) {
                            uint32_t b[4];
                            ldsm4t(vt + r * RB + 16 * swz<RB>(r, 2 * d + hi), b);
                            if constexpr (!k8) {
                                const uint32_t f[4] = {b[0], b[2], b[1], b[3]};
                                mma16816<kMmaBf16>(o[0][d], f, p0, p1);
                            } else {
                                // A piece is 16 dims: the even ones are rows g, the odd ones rows g + 8.
#pragma unroll
                                for (int n = 0; n < 2; ++n) {
                                    const uint32_t f[4] = {codes2<K, 0, 2>(b[2 * n]), codes2<K, 1, 2>(b[2 * n]),
                                                           codes2<K, 0, 2>(b[2 * n + 1]), codes2<K, 1, 2>(b[2 * n + 1])};
                                    mma16816<false>(o[0][2 * d + n], f, p0, p1);
                                }
                            }
                        }
                    }
                } else if (!skip) {
                    // scores
                    float s[MT][2][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
                    if constexpr (!k8) {
                        const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
                        for (int k = 0; k < HD / 16; ++k) {
                            uint32_t b[4];
                            ldsm4(kt + r * RB + 16 * swz<RB>(r, 2 * k + c), b);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                mma16816<kMmaBf16>(s[mt][0], qf[mt][k], b[0], b[1]);
                                mma16816<kMmaBf16>(s[mt][1], qf[mt][k], b[2], b[3]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                            for (int b = 0; b < HD / 64; ++b) {
                                const int r = 8 * nt + g;
                                uint32_t w[4];
                                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                             : "r"(kt + r * RB + 16 * swz<RB>(r, 4 * b + t4))
                                             : "memory");
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t b0 = codes2<K, 0, 1>(w[k]), b1 = codes2<K, 2, 1>(w[k]);
#pragma unroll
                                    for (int mt = 0; mt < MT; ++mt)
                                        mma16816<false>(s[mt][nt], qf[mt][4 * b + k], b0, b1);
                                }
                            }
                    }
                    // scales, mask, running maximum
                    float vs[2][2];        // v's scale of positions (nt, pair) relative to G
                    float vscale[2][2];
                    if constexpr (k8) {
                        float top = 0.f;
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            float2 ks, vv;
                            const uint32_t sa = kt + 2 * S::kTile + 4 * (8 * nt + 2 * t4);
                            asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(ks.x), "=f"(ks.y) : "r"(sa) : "memory");
                            asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(vv.x), "=f"(vv.y) : "r"(sa + 64) : "memory");
                            // Positions that are no keys: whatever stands in the pool there is left out.
                            const int j = key0 + 8 * nt + 2 * t4;
                            vscale[nt][0] = j < t.keys ? vv.x : 0.f;
                            vscale[nt][1] = j + 1 < t.keys ? vv.y : 0.f;
                            top = fmaxf(top, fmaxf(vscale[nt][0], vscale[nt][1]));
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                s[mt][nt][0] *= ks.x;
                                s[mt][nt][1] *= ks.y;
                                s[mt][nt][2] *= ks.x;
                                s[mt][nt][3] *= ks.y;
                            }
                        }
                        const int ne = max(ge, ceil_log2(quad_max(top)));
                        if (ne != ge) {
                            const float down = pow2i(max(ge - ne, -126));
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                for (int d = 0; d < HD / 8; ++d)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[mt][d][e] *= down;
                            ge = ne;
                        }
                        const float inv = pow2i(-ge);
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            vs[nt][0] = vscale[nt][0] * inv;
                            vs[nt][1] = vscale[nt][1] * inv;
                        }
                    }
                    const bool cut = key0 + kStep - 1 > sure || key0 + kStep > t.keys;
                    uint32_t p[MT][4];
                    bool moved = false;
                    float corr[MT][2];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (mt == MT - 1 && h == 1 && !upper) {
                                corr[mt][h] = 1.f;
                                p[mt][h] = p[mt][2 + h] = 0u;
                                continue;
                            }
                            float v[4] = {s[mt][0][2 * h] * rs[mt][h], s[mt][0][2 * h + 1] * rs[mt][h],
                                          s[mt][1][2 * h] * rs[mt][h], s[mt][1][2 * h + 1] * rs[mt][h]};
                            if (cut) {
                                const int last = min(lim[mt][h], t.keys - 1);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (key0 + 8 * (e >> 1) + 2 * t4 + (e & 1) > last) v[e] = -INFINITY;
                            }
                            const float mx = quad_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
                            const float mn = fmaxf(m[mt][h], mx);
                            const float base = mn == -INFINITY ? 0.f : mn;
                            moved |= mn != m[mt][h];
                            corr[mt][h] = ex2(m[mt][h] - base);
                            m[mt][h] = mn;
                            float sum = 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                v[e] = ex2(v[e] - base);
                                sum += v[e];
                            }
                            l[mt][h] = fmaf(l[mt][h], corr[mt][h], sum);
                            if constexpr (k8) {
                                v[0] *= vs[0][0];
                                v[1] *= vs[0][1];
                                v[2] *= vs[1][0];
                                v[3] *= vs[1][1];
                            }
                            p[mt][h] = pack2<kMmaBf16>(v[0], v[1]);
                            p[mt][2 + h] = pack2<kMmaBf16>(v[2], v[3]);
                        }
                    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int d = 0; d < HD / 8; ++d) {
                                o[mt][d][0] *= corr[mt][0];
                                o[mt][d][1] *= corr[mt][0];
                                o[mt][d][2] *= corr[mt][1];
                                o[mt][d][3] *= corr[mt][1];
                            }
                    }
                    // values
                    const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = lane >> 4;
#pragma unroll
                    for (int d = 0; d < RB / 32; ++d) {
                        uint32_t b[4];
                        ldsm4t(vt + r * RB + 16 * swz<RB>(r, 2 * d + c), b);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            if constexpr (!k8) {
                                mma16816<kMmaBf16>(o[mt][2 * d], p[mt], b[0], b[1]);
                                mma16816<kMmaBf16>(o[mt][2 * d + 1], p[mt], b[2], b[3]);
                            } else {
                                // A piece is 16 dims: the even ones make one n tile, the odd ones another.
                                mma16816<false>(o[mt][4 * d], p[mt], codes2<K, 0, 2>(b[0]), codes2<K, 0, 2>(b[1]));
                                mma16816<false>(o[mt][4 * d + 1], p[mt], codes2<K, 1, 2>(b[0]), codes2<K, 1, 2>(b[1]));
                                mma16816<false>(o[mt][4 * d + 2], p[mt], codes2<K, 0, 2>(b[2]), codes2<K, 0, 2>(b[3]));
                                mma16816<false>(o[mt][4 * d + 3], p[mt], codes2<K, 1, 2>(b[2]), codes2<K, 1, 2>(b[3]));
                            }
                        }
                    }
                }
                __syncwarp();
                stage = stage + 1 == S::kStages ? 0 : stage + 1;
            }
            // ---- the four warps meet ----------------------------------------------
#pragma unroll
            for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float sum = kCols ? col_sum(l[mt][h]) : quad_sum(l[mt][h]);
                    const int r = kCols ? 2 * t4 + h : 16 * mt + 8 * h + g;
                    if ((kCols ? g : t4) == 0) {
                        meet.m[warp][r] = m[mt][h];
                        meet.l[warp][r] = sum;
                    }
                }
            __syncthreads();
            float f_row[kM][2];
#pragma unroll
            for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = kCols ? 2 * t4 + h : 16 * mt + 8 * h + g;
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, meet.m[w][r]);
                    f_row[mt][h] = ex2(m[mt][h] - (top == -INFINITY ? 0.f : top));
                    if constexpr (k8) f_row[mt][h] *= pow2i(ge);
                }
            // Four turns, in each of which a warp adds a quarter of its dims, another
            // than the other warps: every element in an order of its own, but a fixed one.
#pragma unroll 1
            for (int turn = 0; turn < kWarps; ++turn) {
#pragma unroll
                for (int d = 0; d < kTiles; d += kCols ? 1 : 2) {
                    int part = (warp + turn) & 3;
                    asm volatile("" : "+r"(part));   // else the branches become an index, and o goes to local memory
                    if (part != d / (kTiles / 4)) continue;
#pragma unroll
                    for (int mt = 0; mt < kM; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float f = f_row[mt][h];
                            if constexpr (kCols) {
                                float2* at = reinterpret_cast<float2*>(&meet.o[2 * t4 + h][16 * d + 2 * g]);
                                float2 v = make_float2(o[mt][d][h] * f, o[mt][d][2 + h] * f);
                                if (turn) {
                                    const float2 was = *at;
                                    v.x += was.x;
                                    v.y += was.y;
                                }
                                *at = v;
                            } else {
                                float4* at = reinterpret_cast<float4*>(&meet.o[16 * mt + 8 * h + g][8 * d + 4 * t4]);
                                const float x0 = o[mt][d][2 * h] * f, x1 = o[mt][d][2 * h + 1] * f;
                                const float y0 = o[mt][d + 1][2 * h] * f, y1 = o[mt][d + 1][2 * h + 1] * f;
                                float4 v = k8 ? make_float4(x0, y0, x1, y1) : make_float4(x0, x1, y0, y1);
                                if (turn) {
                                    const float4 was = *at;
                                    v.x += was.x;
                                    v.y += was.y;
                                    v.z += was.z;
                                    v.w += was.w;
                                }
                                *at = v;
                            }
                        }
                }
                __syncthreads();
            }
            // ---- out: finished rows, or a partial ------------------------------------
            const PartPlace place = part_place(t);
            const bool whole = place.whole;
            const int slot = place.slot;
            if (!whole && place.begins) {
                open = true;
                if (threadIdx.x == 0) note_open<kCost>(a, work, t);
            }
            for (int e = threadIdx.x; e < kRows * (HD / 8); e += kThreads) {
                const int r = e / (HD / 8), c = e % (HD / 8);
                const int i = packed0 + r;
                if (i >= packed) continue;
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, meet.m[w][r]);
                const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sum += meet.l[w][r] * ex2(meet.m[w][r] - base);
                float4 x0, x1;
                if constexpr (k8) {
                    x0 = *reinterpret_cast<const float4*>(&meet.o[r][8 * c]);
                    x1 = *reinterpret_cast<const float4*>(&meet.o[r][8 * c + 4]);
                } else if constexpr (kCols) {
                    const float* from = &meet.o[r][16 * (c >> 1) + (c & 1)];
                    x0 = make_float4(from[0], from[2], from[4], from[6]);
                    x1 = make_float4(from[8], from[10], from[12], from[14]);
                } else {
                    const float* from = &meet.o[r][16 * (c >> 1) + 2 * (c & 1)];
                    float2 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const float2*>(from + 4 * j);
                    x0 = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
                    x1 = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
                }
                if (whole) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const int row = t.q.q0 + i / a.group, qh = t.head * a.group + i % a.group;
                    *reinterpret_cast<uint4*>(a.out.data + (long long)row * a.out.row_bytes +
                                              (long long)qh * a.out.head_bytes + 16 * c) =
                        make_uint4(pack2<BF16>(x0.x * inv, x0.y * inv), pack2<BF16>(x0.z * inv, x0.w * inv),
                                   pack2<BF16>(x1.x * inv, x1.y * inv), pack2<BF16>(x1.z * inv, x1.w * inv));
                    if (a.lse && c == 0)
                        a.lse[(long long)row * a.n_head + qh] =
                            sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
                } else {
                    float* po = a.parts.o + ((long long)slot * kRows + r) * HD + 8 * c;
                    reinterpret_cast<float4*>(po)[0] = x0;
                    reinterpret_cast<float4*>(po)[1] = x1;
                    if (c == 0) {
                        a.parts.ml[(long long)slot * 2 * kRows + r] = top;
                        a.parts.ml[(long long)slot * 2 * kRows + kRows + r] = sum;
                    }
                }
            }
            __syncthreads();
            next_tile<kUnit, kCost>(a, work, t);
            if (t.n <= 0) break;
        }
        cp_wait<0>();
    }
    if (!open && threadIdx.x == 0) a.parts.info[blockIdx.x].n = 0;
}

// What the join takes: the partials of the few-rows kernel's CTAs and of the
// tensor-core kernel's (either may be absent).
struct JoinArgs {
    Rows out;
    float* lse;
    int n_head, group;
    Parts parts[2];
    int n_cta[2];
};

// Adds up the tile that a CTA left open: its slot 1 and the slots 0 of the
// CTAs after it.  kFewShare blocks share the tile of a CTA of the few-rows
// kernel, kTcShare that of one of the tensor-core kernel (up to 256 rows: a
// tile in up to four parts is one round of loads).  HD / 4 threads take a row,
// four dims each; with many parts (a long sequence alone) four such groups
// share a row's parts.  The kernel is a chain of latencies (which tile, its
// maxima, its rows): every load of a step is issued before the first is used,
// and the grid is small, since most CTAs left nothing open (7,296 blocks that
// only look cost 6 us, 912 less than 2).
constexpr int kFewShare = 2, kTcShare = 16;

// One joined row's four dims, and by the first of its threads the row's lse.
template <bool BF16>
__device__ __forceinline__ void put_joined(const JoinArgs& a, const PartInfo& info, int r, int d, float4 acc, float top,
                                           float sum) {
    const int i = info.packed0 + r;
    const int row = info.q0 + i / a.group, qh = info.head * a.group + i % a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(a.out.data + (long long)row * a.out.row_bytes + (long long)qh * a.out.head_bytes + 8 * d) =
        make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
    if (a.lse && d == 0)
        a.lse[(long long)row * a.n_head + qh] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// The rows first, first + step, ... of a tile cut in n <= P parts, R of them at a time.
template <int HD, bool BF16, int P, int R>
__device__ __forceinline__ void join_rows(const JoinArgs& a, const Parts& parts, const PartInfo& info, int c0, int n,
                                          int first, int step, int d, int d_step, int r_step) {
    const int rows = parts.rows, live = info.packed_end - info.packed0;
    for (int r0 = first; r0 < live; r0 += R * step) {
        float m[R][P], l[R][P];
        float4 o[R][P];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const int r = r0 + j * step;
                m[j][k] = -INFINITY;
                l[j][k] = 0.f;
                o[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < live && k < n) {
                    const long long slot = k == 0 ? 2 * c0 + 1 : 2 * (c0 + k);
                    m[j][k] = parts.ml[slot * 2 * rows + r];
                    l[j][k] = parts.ml[(slot * 2 + 1) * rows + r];
                    o[j][k] = reinterpret_cast<const float4*>(parts.o + slot * rows * HD)[d * d_step + r * r_step];
                }
            }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int r = r0 + j * step;
            if (r >= live) break;
            float top = m[j][0];
#pragma unroll
            for (int k = 1; k < P; ++k) top = fmaxf(top, m[j][k]);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const float w = ex2(m[j][k] - base);
                sum = fmaf(l[j][k], w, sum);
                acc.x = fmaf(o[j][k].x, w, acc.x);
                acc.y = fmaf(o[j][k].y, w, acc.y);
                acc.z = fmaf(o[j][k].z, w, acc.z);
                acc.w = fmaf(o[j][k].w, w, acc.w);
            }
            put_joined<BF16>(a, info, r, d, acc, top, sum);
        }
    }
}

// kTc: the tensor-core kernel ran too (the few-rows kernel's tiles alone do not
// need the code for its larger ones: half a microsecond of instruction fetches).
template <int HD, bool BF16, bool kTc>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ JoinArgs a) {
    constexpr int kT = HD / 4, kGroups = 256 / kT, kAhead = 8;
    __shared__ float4 so[256];
    __shared__ float sm_[kGroups], sl[kGroups];
    pdl_launch_dependents();
    pdl_wait();
    int which = 0, c0 = blockIdx.x, y = blockIdx.y, ny = kFewShare;
    if constexpr (kTc) {
        const int few_blocks = kFewShare * a.n_cta[0];
        which = (int)blockIdx.x >= few_blocks;
        ny = which ? kTcShare : kFewShare;
        const int at = blockIdx.x - (which ? few_blocks : 0);
        c0 = at / ny;
        y = at % ny;
    }
    const Parts& parts = a.parts[which];
    const PartInfo info = parts.info[c0];
    if (info.n == 0) return;
    // Neighbouring threads take neighbouring dims or rows, as the partials lie.
    const int g = kTc && parts.beside ? threadIdx.x % kGroups : threadIdx.x / kT;
    const int d = kTc && parts.beside ? threadIdx.x / kGroups : threadIdx.x % kT;
    const int g_step = kTc && parts.beside ? 1 : kT;              // threads from a group to the next
    const int rows = parts.rows, n = min(info.n, a.n_cta[which] - c0);
    const int d_step = kTc && parts.beside ? rows : 1, r_step = kTc && parts.beside ? 1 : kT;
    if constexpr (kTc) {
        // Tiles cut in a few parts: the loads of several rows at a time.
        if (n <= 2) {
            // Half the blocks do: with all of them a prompt's join took 20 us instead of 15.
            if (y < ny / 2)
                join_rows<HD, BF16, 2, 4>(a, parts, info, c0, n, kGroups * y + g, kGroups * (ny / 2), d, d_step, r_step);
            return;
        }
        if (n <= 4)
            return join_rows<HD, BF16, 4, 2>(a, parts, info, c0, n, kGroups * y + g, kGroups * ny, d, d_step, r_step);
    }
    const int share = n > kAhead ? 4 : 1;                  // groups per row
    const int sub = g % share;
    const int at_once = kGroups / share;
    // Every thread takes every turn (the barriers below).
    for (int r0 = y * at_once; info.packed0 + r0 < info.packed_end; r0 += ny * at_once) {
        const int r = r0 + g / share;
        const bool in = info.packed0 + r < info.packed_end;
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) {
            for (int k0 = sub; k0 < n; k0 += kAhead * share) {
                float m[kAhead], l[kAhead];
                float4 o[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int k = k0 + i * share;
                    m[i] = -INFINITY;
                    l[i] = 0.f;
                    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < n) {
                        const long long slot = k == 0 ? 2 * c0 + 1 : 2 * (c0 + k);
                        m[i] = parts.ml[slot * 2 * rows + r];
                        l[i] = parts.ml[(slot * 2 + 1) * rows + r];
                        o[i] = reinterpret_cast<const float4*>(parts.o + slot * rows * HD)[d * d_step + r * r_step];
                    }
                }
                float t = top;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) t = fmaxf(t, m[i]);
                const float base = t == -INFINITY ? 0.f : t, old = ex2(top - base);
                top = t;
                sum *= old;
                acc.x *= old;
                acc.y *= old;
                acc.z *= old;
                acc.w *= old;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float w = ex2(m[i] - base);
                    sum = fmaf(l[i], w, sum);
                    acc.x = fmaf(o[i].x, w, acc.x);
                    acc.y = fmaf(o[i].y, w, acc.y);
                    acc.z = fmaf(o[i].z, w, acc.z);
                    acc.w = fmaf(o[i].w, w, acc.w);
                }
            }
        }
        if (share > 1) {
            so[threadIdx.x] = acc;
            if (d == 0) {
                sm_[g] = top;
                sl[g] = sum;
            }
            __syncthreads();
            const int first = g - sub;
            float t = -INFINITY;
            for (int i = 0; i < share; ++i) t = fmaxf(t, sm_[first + i]);
            const float base = t == -INFINITY ? 0.f : t;
            top = t;
            sum = 0.f;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = 0; i < share; ++i) {
                const float w = ex2(sm_[first + i] - base);
                const float4 o = so[threadIdx.x + (i - sub) * g_step];
                sum = fmaf(sl[first + i], w, sum);
                acc.x = fmaf(o.x, w, acc.x);
                acc.y = fmaf(o.y, w, acc.y);
                acc.z = fmaf(o.z, w, acc.z);
                acc.w = fmaf(o.w, w, acc.w);
            }
            __syncthreads();
        }
        if (!in || sub) continue;
        put_joined<BF16>(a, info, r, d, acc, top, sum);
    }
}

// CTAs of the few-rows kernel: as many as stay resident (ctas_of by the
// registers; shared memory may allow fewer).
constexpr int kMaxCtasPerSm = 4;

template <int HD, Kind K, bool BF16, int MT>
cudaError_t launch_few(AttnArgs& a, int* grid, int n_sm, cudaStream_t st) {
    using S = Shape<HD, K>;
    const size_t smem = (sizeof(Meet<HD, MT>) + 127) / 128 * 128 + kWarps * S::kRing + 8 * ((size_t)a.b.n_seq + 1);
    auto kern = k_paged_attn<HD, K, BF16, MT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    const int by_smem = (int)(228 * 1024 / (smem + 1024));
    *grid = n_sm * max(1, min(by_smem, ctas_of<MT>));
    // No more CTAs than the batch can have units (one, which looks the batch over, if max_q is 0).
    const long long tiles = ((long long)a.b.max_q * a.group + a.tile - 1) / a.tile;
    const long long units = (((long long)a.b.max_pages << a.kv.page_shift) + kUnit - 1) / kUnit;
    if (a.b.n_seq * tiles * a.kv.n_kv < *grid)
        *grid = (int)max(1ll, min((long long)*grid, a.b.n_seq * tiles * a.kv.n_kv * units));
    a.parts = carve_parts(a.parts.info, *grid, rows_of<MT>, false);
    kern<<<*grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <int HD, Kind K, bool BF16>
cudaError_t launch_rows(AttnArgs& a, int* grid, int n_sm, cudaStream_t st) {
    if (a.tile == 8) return launch_few<HD, K, BF16, 0>(a, grid, n_sm, st);
    return a.tile == 16 ? launch_few<HD, K, BF16, 1>(a, grid, n_sm, st) : launch_few<HD, K, BF16, 2>(a, grid, n_sm, st);
}

template <int HD, bool BF16>
cudaError_t launch_kind(AttnArgs& a, int format, int* grid, int n_sm, cudaStream_t st) {
    if (format == QWEN2_KV_INT8) return launch_rows<HD, kInt8, BF16>(a, grid, n_sm, st);
    if (format == QWEN2_KV_E4M3) return launch_rows<HD, kE4m3, BF16>(a, grid, n_sm, st);
    return launch_rows<HD, kSame16, BF16>(a, grid, n_sm, st);
}

template <int HD>
cudaError_t launch_join(const JoinArgs& j, bool bf16, bool tc, cudaStream_t st) {
    const dim3 block(256);
    const dim3 grid = tc ? dim3(kFewShare * j.n_cta[0] + kTcShare * j.n_cta[1]) : dim3(j.n_cta[0], kFewShare);
    if (tc)
        return bf16 ? launch_pdl(k_attn_join<HD, true, true>, grid, block, 0, st, j)
                    : launch_pdl(k_attn_join<HD, false, true>, grid, block, 0, st, j);
    return bf16 ? launch_pdl(k_attn_join<HD, true, false>, grid, block, 0, st, j)
                : launch_pdl(k_attn_join<HD, false, false>, grid, block, 0, st, j);
}

// Which kernels a call needs.  Sequences of up to 32 packed rows are the
// few-rows kernel's, longer ones the tensor-core kernel's; where a batch may
// have both, the few-rows kernel keeps to 16 rows.
struct Plan {
    int tile;            // packed rows of the few-rows kernel's tiles; 0: not launched
    int few;             // most packed rows of its sequences
    bool tc;
};
Plan plan_of(const Batch& b, const Pool& kv, int n_head, bool tensor) {
    const int group = n_head / kv.n_kv;
    const long long most = (long long)b.max_q * group;
    if (most <= 8) return {8, 0x7fffffff, false};
    if (most <= 16) return {16, 0x7fffffff, false};
    if (most <= 32 || !tensor) return {32, 0x7fffffff, false};
    if (b.n_seq == 1) return {0, 0, true};
    return {16, 16, true};
}
bool tensor_kernel(float scale) {
    // Masked scores are -inf before the scale: it has to be positive there.
    return scale > 0.f;
}

}  // namespace

long long attn_workspace(const Batch& b, const Pool& kv, int head_dim, int n_head, int n_sm) {
    const int group = n_head / kv.n_kv;
    const long long most = (long long)b.max_q * group;
    // For either choice of kernels.
    return parts_bytes(n_sm * kMaxCtasPerSm, most <= 8 ? 8 : most <= 16 ? 16 : 32, head_dim) +
           (most > 32 ? parts_bytes(n_sm, tc_tile_rows(group), head_dim) : 0);
}

cudaError_t enqueue_attention(const Pool& kv, const Batch& b, const AttnCall& c, const Rows& q, const Rows& out,
                              int n_sm, cudaStream_t st) {
    AttnArgs a{};
    a.kv = kv;
    a.b = b;
    a.q = q;
    a.out = out;
    a.lse = c.lse;
    a.n_head = c.n_head;
    a.group = c.n_head / kv.n_kv;
    a.causal = c.causal;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    const bool bf16 = c.dtype == QWEN2_DTYPE_BF16;
    TcMaps maps;
    Plan plan = plan_of(b, kv, c.n_head, tensor_kernel(c.scale));
    if (plan.tc && !tc_encode(maps, kv, c, q, b.n_rows)) plan = plan_of(b, kv, c.n_head, false);
    JoinArgs j{};
    j.out = out;
    j.lse = c.lse;
    j.n_head = c.n_head;
    j.group = a.group;
    cudaError_t e = cudaSuccess;
    char* ws = static_cast<char*>(c.workspace);
    if (plan.tile) {
        a.tile = plan.tile;
        a.rows_lo = 0;
        a.rows_hi = plan.few;
        a.parts.info = reinterpret_cast<PartInfo*>(ws);
        int* g = &j.n_cta[0];
        if (c.head_dim == 64) e = bf16 ? launch_kind<64, true>(a, c.format, g, n_sm, st) : launch_kind<64, false>(a, c.format, g, n_sm, st);
        else e = bf16 ? launch_kind<128, true>(a, c.format, g, n_sm, st) : launch_kind<128, false>(a, c.format, g, n_sm, st);
        if (e != cudaSuccess) return e;
        j.parts[0] = a.parts;
        ws += parts_bytes(j.n_cta[0], plan.tile, c.head_dim);
    }
    if (plan.tc) {
        a.tile = tc_tile_rows(a.group);
        a.rows_lo = plan.tile ? plan.few : 0;
        a.rows_hi = 0x7fffffff;
        a.parts = carve_parts(ws, n_sm, a.tile, true);
        e = enqueue_attention_tc(maps, a, c.format, c.head_dim, bf16, n_sm, plan.tile != 0, st);
        if (e != cudaSuccess) return e;
        j.parts[1] = a.parts;
        j.n_cta[1] = n_sm;
    }
    return c.head_dim == 64 ? launch_join<64>(j, bf16, plan.tc, st) : launch_join<128>(j, bf16, plan.tc, st);
}

}  // namespace paged
}  // namespace qwen2
