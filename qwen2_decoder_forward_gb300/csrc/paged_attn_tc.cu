// Attention over the paged cache for chunks and prompts: the products on
// tcgen05, the queries and 16-bit pages by TMA, 8-bit pages through registers.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = 2^(s_ij - m_i),
//   s_ij = scale log2(e) q_i . k_j,
//
// one pass over the keys with a running reference m_i of each row: any m_i
// gives the same quotient, so m_i is moved up to the row's maximum (and the
// accumulator rescaled) only when that has grown by more than 2^8 since; the
// weights then stay below 2^8, far inside f16, and rescales are rare.
//
// A CTA (one per SM, persistent over its part of the work list, paged.cuh)
// takes a tile of two 128-row halves A and B that share every K and V tile:
// each half is R = 128 / group rows of the sequence with the group's heads
// packed (a TMA box [R][group][64] lands as consecutive 128-byte rows), so a
// K / V tile is read once for 2 R rows of all the group's heads.  Per unit of
// 128 positions and half:  S = Q K^T into 128 columns of TMEM;
// thread i of the half's warpgroup owns row i,
// takes S into registers, writes P = 2^(s - m) as 16-bit pairs back to TMEM,
// and the tensor core takes P from there: O += P V.  While the warpgroup of
// one half is at its softmax, the products of the other half run.
//
// Warps: 0-3 softmax of A, 4-7 of B, 8 and 10 issue the products of A and B
// (waits and commits cost an issuing thread some 150 cycles each, one thread
// for both halves left the tensor pipe idle half the time), 9 feeds (11 fills
// the third warpgroup).  TMEM (512 columns): S_A, S_B at 0 and 128; O_A, O_B
// from 256.  head_dim 64 has columns of their own for P, so S of the next unit
// is made while P of this one is; for head_dim 128 P lies over its own S and S
// of the next unit follows P V.  P is handed over in two parts of 64 positions.
//
// 8-bit pages: four more warps (12-15) read the codes, widen them to exact
// 16-bit values (of the queries' type) and store the swizzled tiles that TMA
// would have written.  The scales stay out of the products: k's multiplies the
// scores, v's the probabilities, relative to G, the largest v scale so far
// rounded up to a power of two, which O carries like the reference m.
//
// V is the [position][dim] tile as it lies in the pages: an MN-major B
// operand, so nothing is transposed.  Positions of the last unit that are no
// keys are zeroed in V (0 * NaN) and masked in S.
#include <cuda.h>
#include <cuda_fp8.h>

#include "paged.cuh"
#include "paged.h"
#include "sm100.cuh"
#include "tmap.h"

namespace qwen2 {
namespace paged {

namespace {

using namespace sm100;

constexpr int kUnit = 128;                 // positions per unit
constexpr int kCost = 2;                   // slots of a tile beside its units (paged.cuh)
enum Kind { kSame16, kInt8, kE4m3 };
// Registers per thread (setmaxnreg): a softmax thread holds a row of S.
// 16-bit pages: 384 threads launched with 168 (64,512 in all),
// 2 * 128 * 200 + 128 * 104 = 64,512.  8-bit pages: 512 threads launched with
// 128 (65,536), 2 * 128 * 184 + 2 * 128 * 72 = 65,536.
template <Kind K>
struct Split {
    static constexpr int kThreads = K == kSame16 ? 384 : 512;
    static constexpr int kSoftmax = K == kSame16 ? 200 : 184;
    static constexpr int kOther = K == kSame16 ? 104 : 72;
};
constexpr int kFeeders = 4;                // warps that widen 8-bit codes
constexpr int kStaging = 8 * 2048;         // output rows on their way, 2 KB per softmax warp
constexpr int kScaleUnits = 4;             // units whose scales are kept (8-bit pages)
constexpr int kMaxStages = 12, kMaxStages8 = 6;
constexpr int kHalfBytes = 128 * 128;      // 128 rows of 64 16-bit elements
constexpr uint32_t kTmemCols = 512;
constexpr float kSlack = 8.f;              // log2 of the growth that is left in the weights

struct TcSmem {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full, q_empty, s_full[2], s_read[2], p_lo[2], p_hi[2], o_full[2], turn[2], tail, drain[2];
    unsigned bad[8];                       // per unit (mod 8): its positions in bad pages, 16 per bit
    int g[kScaleUnits];                    // 8-bit pages, per unit (mod 4): log2 of G
    uint32_t tmem_slot;
    int abort;
};
constexpr int kHead = 1024;                // TcSmem, in front of the 1024-byte aligned tiles
static_assert(sizeof(TcSmem) <= kHead - 64, "");      // the last 64 bytes: the feeders' reduction

struct TcArgs {
    AttnArgs a;
    int sub;              // packed rows of a half: R * group
    int sub_rows;         // R
    int stages;           // ring stages of one K or V tile
    int kv_rank[3];       // tensor-map dims (1..3) of position, head, page
    int min_slots;
};

// Waits for the phase of parity `parity`, at most about kWaitNs: the SM's own
// clock is read (a read of the global timer costs a large part of a unit's
// time).  False once this or another wait of the block has given up.
constexpr long long kWaitClocks = (long long)kWaitNs * 2;      // 2 s or more at up to 2 GHz
__device__ __forceinline__ bool wait_slow(uint64_t* bar, unsigned parity, TcSmem& sm, int* guard) {
    const long long t0 = clock64();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
        if (clock64() - t0 > kWaitClocks) {
            sm.abort = 1;
            raise_guard(guard, kGuardTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait(uint64_t* bar, unsigned parity, TcSmem& sm, int* guard) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, sm, guard);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// Descriptor of a V tile as B operand with N = dims contiguous (MN-major,
// 128-byte swizzle): 64-dim halves kHalfBytes apart (leading offset), groups
// of 8 positions 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t desc_mn128(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kHalfBytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// kind::f16 instruction descriptor: f32 accumulator, A and B f16 or bf16, B
// K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc16(int M, int N, bool bf16, bool b_mn) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] . B[smem], issued by one thread.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 columns of this thread's TMEM lane, without waiting for them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's TMEM loads; no use of `r` moves above it.
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void pin32(uint32_t (&r)[32]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]));
    asm volatile("" : "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                      "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]));
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A place in the ring of K and V tiles: entries are stored and used in order.
struct Cursor {
    unsigned stage = 0, round = 0;
    __device__ __forceinline__ void next(unsigned stages) {
        if (++stage == stages) {
            stage = 0;
            ++round;
        }
    }
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int HD>
struct Tmem {
    static constexpr uint32_t s(int x) { return 128u * x; }
    static constexpr uint32_t o(int x) { return 256u + (uint32_t)HD * x; }
    static constexpr uint32_t p(int x) { return HD == 64 ? 384u + 64u * x : s(x); }
};

// a * b + c on two floats at once.
__device__ __forceinline__ void fma2(float& x, float& y, float b, float c) {
    asm("{\n\t.reg .b64 p, q, r;\n\t"
        "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}

// Scores of 32 positions times k's scales.
__device__ __forceinline__ void scale_scores(uint32_t (&s)[32], uint32_t at) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const float4 ks = lds4(at + 4 * e);
        float y[4] = {__uint_as_float(s[e]), __uint_as_float(s[e + 1]), __uint_as_float(s[e + 2]),
                      __uint_as_float(s[e + 3])};
        mul2(y[0], y[1], ks.x, ks.y);
        mul2(y[2], y[3], ks.z, ks.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[e + i] = __float_as_uint(y[i]);
    }
}
__device__ __forceinline__ void top2(float& v, uint32_t a, uint32_t b) {
    v = max3(v, __uint_as_float(a), __uint_as_float(b));
}
// Two scores to weights, in place: 2^(score * scale + base).
__device__ __forceinline__ void weigh2(uint32_t& a, uint32_t& b, float scale, float base) {
    float y = __uint_as_float(a), z = __uint_as_float(b);
    fma2(y, z, scale, base);
    a = __float_as_uint(ex2(y));
    b = __float_as_uint(ex2(z));
}

// 64 bytes of each of the warp's 32 rows (lane l holds row l's, dst its
// address, null for a row that is not written) to offset `off` of the rows.
__device__ __forceinline__ void put_rows64(uint32_t stage, const uint32_t (&w)[16], char* dst, int off, int lane) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)),
                     "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                     : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2), j = lane & 3;
        char* to = reinterpret_cast<char*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(stage + r * 64 + ((j ^ (r >> 1 & 3)) << 4))
                     : "memory");
        if (to) *reinterpret_cast<uint4*>(to + off + 16 * j) = v;
    }
}

// 16 codes as 16-bit values, in order; exact.
template <Kind K, bool BF16>
__device__ __forceinline__ void widen16(const uint4& raw, uint32_t (&o)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (K == kInt8 && !BF16) {
                // 1024 + (c + 128), minus 1152.
                const uint32_t h = __byte_perm(w[i] ^ 0x80808080u, 0x64646464u, j ? 0x4342 : 0x4140);
                const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
                o[2 * i + j] = *reinterpret_cast<const uint32_t*>(&v);
            } else if constexpr (K == kInt8) {
                // c = (128 + its low 7 bits) - (128, or 256 if negative).
                const uint32_t h = __byte_perm(w[i], 0x43434343u, j ? 0x4342 : 0x4140);
                const uint32_t x = h & 0xff7fff7fu, y = h & 0xff80ff80u;
                const __nv_bfloat162 v =
                    __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
                o[2 * i + j] = *reinterpret_cast<const uint32_t*>(&v);
            } else {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
                if constexpr (!BF16) {
                    o[2 * i + j] = (uint32_t)h.x | (uint32_t)h.y << 16;
                } else {
                    const float2 f = __half22float2(__half2(h));
                    o[2 * i + j] = pack2<true>(f.x, f.y);
                }
            }
        }
}

// The power of two at or above v, as an exponent in [-100, 100].
__device__ __forceinline__ int ceil_log2(float v) {
    const int b = __float_as_int(v);
    const int e = ((b >> 23) & 255) - 127 + ((b & 0x7fffff) != 0);
    return min(max(e, -100), 100);
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Barrier of the four feeding warps that tells all of them whether every one
// got through its wait: they go on, or stop, together.
__device__ __forceinline__ bool feeders_agree(bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)ok)
        : "memory");
    return all != 0;
}

template <int HD, bool BF16, Kind K>
__global__ void __launch_bounds__(Split<K>::kThreads, 1)
    k_paged_attn_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcArgs args) {
    using T = Tmem<HD>;
    constexpr int kHalves = HD / 64;
    constexpr int kTileBytes = kHalves * kHalfBytes;
    constexpr bool k8 = K != kSame16;
    constexpr bool kOverlay = HD == 128;        // P lies over S
    const AttnArgs& a = args.a;
    extern __shared__ unsigned char tc_smem_raw[];
    const uint32_t pad = (1024u - (smem_addr(tc_smem_raw) & 1023u)) & 1023u;
    TcSmem& sm = *reinterpret_cast<TcSmem*>(tc_smem_raw + pad);
    const uint32_t q_tiles = smem_addr(&sm) + kHead;                 // A, B
    const uint32_t ring = q_tiles + 2 * kTileBytes;
    const uint32_t staging = ring + args.stages * kTileBytes;        // 2 KB per softmax warp
    const uint32_t scales = staging + kStaging;                      // 8-bit: [kScaleUnits][k, v / G][kUnit] f32
    long long* prefix = reinterpret_cast<long long*>(tc_smem_raw + pad + kHead + (2 + args.stages) * kTileBytes + kStaging +
                                                     (k8 ? kScaleUnits * 2 * kUnit * 4 : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < args.stages; ++i) {
            mbar_init(&sm.full[i], k8 ? kFeeders : 1);
            mbar_init(&sm.empty[i], 2);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sm.s_full[x], 1);
            mbar_init(&sm.s_read[x], 128);
            mbar_init(&sm.p_lo[x], 128);
            mbar_init(&sm.p_hi[x], 128);
            mbar_init(&sm.o_full[x], 1);
            mbar_init(&sm.turn[x], 1);
            mbar_init(&sm.drain[x], 1);
        }
        mbar_init(&sm.tail, 1);
        mbar_init_fence();
        sm.abort = 0;
    }
    if (warp == 8) tmem_alloc(&sm.tmem_slot, kTmemCols);
    if (warp == 9 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        if constexpr (!k8) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
    }
    const WorkList work = build_work<kUnit, kCost>(a, prefix, args.min_slots);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_slot;
    bool open = false;
    if (work.begin < work.end) {
        Tile t = find_tile<kUnit, kCost>(a, work);
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Split<K>::kSoftmax));
            // ---- softmax of half x --------------------------------------------------
            const int x = warp >> 2, rl = 32 * (warp & 3) + lane;
            const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            const uint32_t t_s = lanes + T::s(x), t_o = lanes + T::o(x), t_p = lanes + T::p(x);
            const float sc = a.scale_log2;
            unsigned n_s = 0;          // units of this half so far
            unsigned unit = 0;         // units of the CTA before this tile
            Cursor cur;                // K of the current unit; V follows
            unsigned v_stage = 0;      // V of the unit before
            bool ok = true;
            while (ok) {
                const int packed0 = t.t * a.tile, packed = t.q.n * a.group;
                const int i = packed0 + x * args.sub + rl;
                const bool live = rl < args.sub && i < packed;
                if (packed0 + x * args.sub < packed) {
                    const int lim = live ? min(row_limit(a, t.q, i), t.keys - 1) : t.keys - 1;
                    const int sure = min(row_limit(a, t.q, packed0 + x * args.sub), t.keys - 1);
                    float m = -INFINITY, l0 = 0.f, l1 = 0.f;
                    int g = -100;          // log2 of G
                    for (int u = 0; u < t.n; ++u, ++n_s) {
                        const int key0 = (t.u0 + u) * kUnit;
                        ok = __all_sync(0xffffffffu, wait(&sm.s_full[x], n_s & 1, sm, a.b.guard));
                        if (!ok) break;
                        tc_fence_after();
                        uint32_t s[4][32];
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld32_async(t_s + 32 * c, s[c]);
                        const unsigned bad = sm.bad[(unit + u) & 7];
                        if (rl == 0) {
                            // This half is done with the unit's K tile, with the queries after the
                            // last one, and (S was issued after the last P V had completed) with
                            // the V tile before.
                            mbar_arrive(&sm.empty[cur.stage]);
                            if (u + 1 == t.n) mbar_arrive(&sm.q_empty);
                            if (kOverlay && u > 0) mbar_arrive(&sm.empty[v_stage]);
                        }
                        cur.next(args.stages);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 4; ++c) pin32(s[c]);
                        if constexpr (!kOverlay) {
                            tc_fence_before();
                            mbar_arrive(&sm.s_read[x]);
                        }
                        const uint32_t at = scales + ((unit + u) % kScaleUnits) * (2 * kUnit * 4);
                        if constexpr (k8) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) scale_scores(s[c], at + 128 * c);
                        }
                        // With a reference already there, the weights of the first 64
                        // positions are made against it while the maximum is still being
                        // taken: it has to move only if some score has outgrown it.
                        const bool cut = key0 + kUnit - 1 > sure || bad;
                        const bool ahead = kOverlay && !k8 && u > 0 && !cut && !__any_sync(0xffffffffu, m == -INFINITY);
                        float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        float corr = 1.f;
                        bool moved = false;
                        const auto settle = [&]() {
                            const float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) * sc;
                            const bool move = top > m + kSlack;
                            if (move) {
                                corr = ex2(m - top);
                                m = top;
                                l0 *= corr;
                                l1 *= corr;
                            }
                            moved = __any_sync(0xffffffffu, move);
                        };
                        if (!ahead) {
                            if (cut) {
                                const int last = lim - key0;      // last position of the unit the row sees
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if (__any_sync(0xffffffffu, last < 32 * c + 31)) {
#pragma unroll
                                        for (int e = 0; e < 32; ++e)
                                            if (32 * c + e > last) s[c][e] = 0xff800000u;
                                    }
                                if (bad) {
#pragma unroll
                                    for (int c = 0; c < 8; ++c)
                                        if (bad >> c & 1)
#pragma unroll
                                            for (int e = 0; e < 16; ++e) s[c / 2][16 * (c % 2) + e] = 0xff800000u;
                                }
                            }
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) top2(v[e / 2 & 3], s[c][e], s[c][e + 1]);
                            settle();
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) weigh2(s[c][e], s[c][e + 1], sc, m == -INFINITY ? 0.f : -m);
                        } else {
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    top2(v[e / 2 & 1], s[c][e], s[c][e + 1]);
                                    top2(v[2 + (e / 2 & 1)], s[2 + c][e], s[2 + c][e + 1]);
                                    weigh2(s[c][e], s[c][e + 1], sc, -m);
                                }
                            settle();
                            if (moved) {
                                // The scores are still in TMEM: P has not been stored yet.
#pragma unroll
                                for (int c = 0; c < 2; ++c) tmem_ld32_async(t_s + 32 * c, s[c]);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    pin32(s[c]);
                                    if constexpr (k8) scale_scores(s[c], at + 128 * c);
#pragma unroll
                                    for (int e = 0; e < 32; e += 2) weigh2(s[c][e], s[c][e + 1], sc, -m);
                                }
                            }
                        }
                        bool scale_o = moved;
                        if constexpr (k8) {
                            const int ng = sm.g[(unit + u) % kScaleUnits];
                            corr *= pow2i(max(g - ng, -126));
                            scale_o = scale_o || ng != g;
                            g = ng;
                        }
                        if (u > 0 && (!kOverlay || scale_o)) {
                            // P V of the unit before: P's columns and O are free after it.
                            ok = __all_sync(0xffffffffu, wait(&sm.o_full[x], (n_s - 1) & 1, sm, a.b.guard));
                            if (!ok) break;
                            tc_fence_after();
                            if (!kOverlay && rl == 0) mbar_arrive(&sm.empty[v_stage]);
                        }
                        v_stage = cur.stage;
                        cur.next(args.stages);
                        if (u > 0 && scale_o) {
#pragma unroll 1
                            for (int c = 0; c < HD / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32_async(t_o + 32 * c, o);
                                tmem_ld_wait();
                                pin32(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                                tmem_st32(t_o + 32 * c, o);
                            }
                        }
                        const float base = m == -INFINITY ? 0.f : -m;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t p[32];
                            [[maybe_unused]] float4 vs;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                uint32_t& sy = s[2 * c + e / 16][2 * e % 32];
                                uint32_t& sz = s[2 * c + e / 16][2 * e % 32 + 1];
                                if (c) weigh2(sy, sz, sc, base);
                                float y = __uint_as_float(sy), z = __uint_as_float(sz);
                                add2(l0, l1, y, z);
                                if constexpr (k8) {
                                    if (e % 2 == 0) vs = lds4(at + 4 * kUnit + 4 * (64 * c + 2 * e));
                                    mul2(y, z, e % 2 ? vs.z : vs.x, e % 2 ? vs.w : vs.y);
                                }
                                p[e] = pack2<BF16>(y, z);
                            }
                            tmem_st32(t_p + 32 * c, p);
                            tmem_st_wait();
                            tc_fence_before();
                            mbar_arrive(c ? &sm.p_hi[x] : &sm.p_lo[x]);
                        }
                    }
                    if (!ok) break;
                    // ---- the half's rows ------------------------------------------------
                    ok = __all_sync(0xffffffffu, wait(&sm.o_full[x], (n_s - 1) & 1, sm, a.b.guard));
                    if (!ok) break;
                    tc_fence_after();
                    if (rl == 0) mbar_arrive(&sm.empty[v_stage]);
                    const float l = l0 + l1, unit_g = k8 ? pow2i(g) : 1.f;
                    const PartPlace place = part_place(t);
                    const int slot = place.slot, r = x * args.sub + rl;
                    // Rows go out through the warp's staging buffer: 64 bytes of each of its 32 rows
                    // at a time, written a row per lane and stored four lanes a row (a row per lane
                    // straight to memory touches 32 lines a store and holds the load / store unit
                    // for 5,000 cycles a tile).
                    const bool whole = place.whole;
                    const float f = !whole ? unit_g : l == 0.f ? 0.f : unit_g / l;
                    char* dst;
                    if (whole) {
                        const int row = t.q.q0 + i / a.group, qh = t.head * a.group + i % a.group;
                        dst = a.out.data + (long long)row * a.out.row_bytes + (long long)qh * a.out.head_bytes;
                        if (live && a.lse)
                            a.lse[(long long)row * a.n_head + qh] =
                                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                    } else {
                        dst = reinterpret_cast<char*>(a.parts.o + ((long long)slot * a.parts.rows + r) * HD);
                        if (live) {
                            a.parts.ml[(long long)slot * 2 * a.parts.rows + r] = m;
                            a.parts.ml[((long long)slot * 2 + 1) * a.parts.rows + r] = l;
                        }
                    }
                    if (!live) dst = nullptr;
                    const uint32_t stage = staging + 2048 * warp;
#pragma unroll 1
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_async(t_o + 32 * c, o);
                        tmem_ld_wait();
                        pin32(o);
                        if (whole) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = pack2<BF16>(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
                            put_rows64(stage, w, dst, 64 * c, lane);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            put_rows64(stage, reinterpret_cast<const uint32_t(&)[16]>(o[0]), dst, 128 * c, lane);
                            put_rows64(stage, reinterpret_cast<const uint32_t(&)[16]>(o[16]), dst, 128 * c + 64, lane);
                        }
                    }
                    if (!whole && place.begins) {
                        open = true;
                        if (tid == 0) note_open<kCost>(a, work, t);
                    }
                    tc_fence_before();
                } else {
                    for (int u = 0; u < 2 * t.n; ++u) cur.next(args.stages);
                }
                unit += t.n;
                next_tile<kUnit, kCost>(a, work, t);
                if (t.n <= 0) break;
            }
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<K>::kOther));
        }
        if (warp == 8 || warp == 10) {
            // ---- products of half x ---------------------------------------------------
            if (lane == 0) {
                constexpr uint32_t id_s = idesc16(128, kUnit, BF16, false), id_o = idesc16(128, HD, BF16, true);
                const int x = warp == 8 ? 0 : 1;
                const uint64_t qd = desc_sw128(q_tiles + x * kTileBytes);
                const uint32_t t_s = tmem + T::s(x), t_o = tmem + T::o(x), t_p = tmem + T::p(x);
                unsigned n_u = 0, seg = 0;       // P V products so far; tiles
                unsigned turns = 0;              // units of tiles with both halves so far
                Cursor cur;
                bool ok = true;
                const auto landed = [&](const Cursor& c) {
                    ok = ok && wait(&sm.full[c.stage], c.round & 1, sm, a.b.guard);
                };
                // S against the K tile at `cur`.
                const auto issue_s = [&](bool hand_over) {
                    const uint64_t kd = desc_sw128(ring + cur.stage * kTileBytes);
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) {
                        if (k == HD / 32 && hand_over) mbar_arrive(&sm.turn[x ^ 1]);
                        const uint32_t off = (uint32_t)((k / 4) * kHalfBytes + (k % 4) * 32) >> 4;
                        mma_f16(t_s, qd + off, kd + off, id_s, k != 0 ? 1u : 0u);
                    }
                    mma_commit(&sm.s_full[x]);
                };
                for (;; ++seg) {
                    const bool both = t.t * a.tile + args.sub < t.q.n * a.group;
                    ok = ok && wait(&sm.q_full, seg & 1, sm, a.b.guard);
                    if (x == 1 && !both) {
                        // No rows in this half: its share of releasing the ring all the same.
                        for (int e = 0; e < 2 * t.n && ok; ++e) {
                            landed(cur);
                            if (ok) mbar_arrive(&sm.empty[cur.stage]);
                            cur.next(args.stages);
                        }
                        if (ok) mbar_arrive(&sm.q_empty);
                    } else {
                        landed(cur);
                        if (kOverlay && n_u) ok = ok && wait(&sm.o_full[x], (n_u - 1) & 1, sm, a.b.guard);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(false);
                        cur.next(args.stages);
                        for (int u = 0; u < t.n; ++u) {
                            const Cursor v = cur;              // V of this unit; K of the next one follows
                            const bool more = u + 1 < t.n;
                            cur.next(args.stages);
                            if (!kOverlay) {
                                // S of the next unit once this one's is in registers.
                                ok = ok && wait(&sm.s_read[x], n_u & 1, sm, a.b.guard);
                                if (more) {
                                    landed(cur);
                                    if (!ok) break;
                                    tc_fence_after();
                                    issue_s(false);
                                    cur.next(args.stages);
                                }
                            }
                            landed(v);
                            const uint64_t vd = desc_mn128(ring + v.stage * kTileBytes);
                            // The first 64 positions' P V while the others' P is made.
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                ok = ok && wait(c ? &sm.p_hi[x] : &sm.p_lo[x], n_u & 1, sm, a.b.guard);
                                if (kOverlay && c == 0 && both && (x == 1 || turns))
                                    ok = ok && wait(&sm.turn[x], (x == 1 ? turns : turns - 1) & 1, sm, a.b.guard);
                                if (!ok) break;
                                tc_fence_after();
#pragma unroll
                                for (int k = 4 * c; k < 4 * c + 4; ++k)
                                    mma_ts(t_o, t_p + 8 * k, vd + (2048 * k >> 4), id_o, u > 0 || k > 0 ? 1u : 0u);
                            }
                            if (!ok) break;
                            mma_commit(&sm.o_full[x]);
                            ++n_u;
                            if (kOverlay && more) {
                                landed(cur);
                                ok = ok && wait(&sm.o_full[x], (n_u - 1) & 1, sm, a.b.guard);
                                if (!ok) break;
                                tc_fence_after();
                                // The other half's turn comes with the second part of S: P V and the
                                // next S of one half run together, so that the halves' softmaxes fall
                                // into each other's products.
                                issue_s(both);
                                cur.next(args.stages);
                            }
                            if (kOverlay && both) {
                                if (!more) mbar_arrive(&sm.turn[x ^ 1]);
                                ++turns;
                            }
                        }
                    }
                    next_tile<kUnit, kCost>(a, work, t);
                    if (t.n <= 0 || !ok) break;
                }
                if (!ok) {   // products in flight end before the tensor memory is given back
                    mma_commit(&sm.drain[x]);
                    mbar_wait(&sm.drain[x], 0, kWaitNs);
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---- feed: queries, and 16-bit pages ------------------------------------------
            const int page_rows = 1 << a.kv.page_shift, box = min(page_rows, kUnit), boxes = kUnit / box;
            const int p = lane / kHalves, h = lane % kHalves;
            unsigned seg = 0, unit = 0, n_tail = 0;
            Cursor cur;
            bool ok = true;
            while (ok) {
                const int halves = t.t * a.tile + args.sub < t.q.n * a.group ? 2 : 1;
                if (seg) ok = __all_sync(0xffffffffu, wait(&sm.q_empty, (seg - 1) & 1, sm, a.b.guard));
                if (!ok) break;
                if (lane == 0) {
                    mbar_expect_tx(&sm.q_full, (unsigned)(halves * kHalves * args.sub * 128));
                    for (int x = 0; x < halves; ++x)
                        for (int c = 0; c < kHalves; ++c)
                            tma_load_3d(q_tiles + x * kTileBytes + c * kHalfBytes, &tm_q, 64 * c, t.head * a.group,
                                        t.q.q0 + (2 * t.t + x) * args.sub_rows, &sm.q_full);
                }
                __syncwarp();
                ++seg;
                for (int u = 0; !k8 && u < t.n && ok; ++u, ++unit) {
                    const int key0 = (t.u0 + u) * kUnit, key = key0 + p * box;
                    int page = -1;
                    bool is_bad = false;
                    if (p < boxes && key < t.keys) {
                        page = __ldg(a.b.pages + (long long)t.s * a.b.pages_stride + (key >> a.kv.page_shift));
                        if ((unsigned)page >= (unsigned)a.kv.n_pages) {
                            is_bad = true;
                            page = -1;
                            raise_guard(a.b.guard, QWEN2_GUARD_PAGE);
                        }
                    }
                    const unsigned bad = __reduce_or_sync(
                        0xffffffffu, is_bad ? ((1u << (box / 16)) - 1) << (p * box / 16) : 0u);
                    const unsigned bytes = (unsigned)(__popc(__ballot_sync(0xffffffffu, page >= 0)) * box * 128);
                    const bool whole = key0 + kUnit <= t.keys && !bad;
                    int at[3];
                    at[args.kv_rank[0]] = key & (page_rows - 1);
                    at[args.kv_rank[1]] = t.head;
                    at[args.kv_rank[2]] = page;
                    for (int kv = 0; kv < 2 && ok; ++kv, cur.next(args.stages)) {
                        const unsigned st = cur.stage, round = cur.round;
                        if (round) ok = __all_sync(0xffffffffu, wait(&sm.empty[st], (round - 1) & 1, sm, a.b.guard));
                        if (!ok) break;
                        const uint32_t tile = ring + st * kTileBytes;
                        uint64_t* bar = kv && !whole ? &sm.tail : &sm.full[st];
                        if (lane == 0) {
                            if (!kv) sm.bad[unit & 7] = bad;
                            mbar_expect_tx(bar, bytes);
                        }
                        __syncwarp();
                        if (page >= 0)
                            tma_load_4d(tile + h * kHalfBytes + p * box * 128, kv ? &tm_v : &tm_k, 64 * h, at[0], at[1],
                                        at[2], bar);
                        if (kv && !whole) {
                            // Positions that are no keys: zeros in V.
                            ok = __all_sync(0xffffffffu, wait(&sm.tail, n_tail & 1, sm, a.b.guard));
                            ++n_tail;
                            if (!ok) {
                                mbar_wait(&sm.tail, (n_tail - 1) & 1, kWaitNs);
                                break;
                            }
                            // Eight lanes a 128-byte row, four rows a store.
                            for (int r = (bad ? 0 : max(0, t.keys - key0) & ~3) + (lane >> 3); r < kUnit; r += 4)
                                if (key0 + r >= t.keys || (bad >> (r / 16) & 1))
#pragma unroll
                                    for (int c = 0; c < kHalves; ++c)
                                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                         tile + c * kHalfBytes + r * 128 + (lane & 7) * 16),
                                                     "r"(0)
                                                     : "memory");
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sm.full[st]);
                        }
                    }
                }
                next_tile<kUnit, kCost>(a, work, t);
                if (t.n <= 0 || !ok) break;
            }
            if (!ok && !k8) {   // copies in flight land before the shared memory is given back
                for (unsigned st = 0; st < (unsigned)args.stages; ++st)   // each stage's last entry
                    if (st < cur.stage || cur.round)
                        mbar_wait(&sm.full[st], (st < cur.stage ? cur.round : cur.round - 1) & 1, kWaitNs);
            }
            if (!ok) {
                if (seg) mbar_wait(&sm.q_full, (seg - 1) & 1, kWaitNs);
            }
            __syncwarp();
        } else if (k8 && warp >= 12) {
            // ---- feed: 8-bit pages ------------------------------------------------------
            // Thread e takes 16-byte piece e % 4 of row e / 4 (+ 32 rows a step) of
            // each 64-dim half: two adjacent rows' pieces fill all banks.
            const int e0 = tid - 384, piece = e0 & 3, row0 = e0 >> 2;
            constexpr int kPieces = 4 * kHalves;        // per thread and tile
            unsigned unit = 0;
            Cursor cur;
            bool ok = true, stop = false;
            while (!stop) {
                int g = -100;
                for (int u = 0; u < t.n; ++u, ++unit) {
                    const int key0 = (t.u0 + u) * kUnit;
                    // Lane l holds the page of positions 16 (l % 8) .. of the unit.
                    const int key_l = key0 + 16 * (lane & 7);
                    int page_l = -1;
                    bool is_bad = false;
                    if (key_l < t.keys) {
                        page_l = __ldg(a.b.pages + (long long)t.s * a.b.pages_stride + (key_l >> a.kv.page_shift));
                        if ((unsigned)page_l >= (unsigned)a.kv.n_pages) {
                            is_bad = true;
                            page_l = -1;
                            raise_guard(a.b.guard, QWEN2_GUARD_PAGE);
                        }
                    }
                    const unsigned bad = __ballot_sync(0xffffffffu, is_bad) & 0xffu;
                    // This thread's rows: row0 + 32 j, j = 0 .. 3.
                    long long src[4];
                    bool in[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = row0 + 32 * j, pg = __shfl_sync(0xffffffffu, page_l, r >> 4);
                        in[j] = pg >= 0 && key0 + r < t.keys;
                        src[j] = in[j] ? (long long)pg * a.kv.page_bytes +
                                             (long long)((key0 + r) & ((1 << a.kv.page_shift) - 1)) * a.kv.token_bytes +
                                             (long long)t.head * a.kv.head_bytes + 16 * piece
                                       : 0;
                    }
                    // Position e0's scales.
                    const int pg_s = __shfl_sync(0xffffffffu, page_l, (e0 >> 4) & 7);
                    float ks = 0.f, vs = 0.f;
                    if (pg_s >= 0 && key0 + e0 < t.keys) {
                        const long long i = (((long long)pg_s * a.kv.n_kv + t.head) << a.kv.page_shift) +
                                            ((key0 + e0) & ((1 << a.kv.page_shift) - 1));
                        ks = __ldg(a.kv.k_scale + i);
                        vs = __ldg(a.kv.v_scale + i);
                    }
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const char* base = kv ? a.kv.v : a.kv.k;
                        uint4 raw[kPieces];
#pragma unroll
                        for (int i = 0; i < kPieces; ++i)
                            raw[i] = in[i & 3] ? ld_stream_v4(base + src[i & 3] + 64 * (i >> 2))
                                               : make_uint4(0, 0, 0, 0);
                        const unsigned st = cur.stage, round = cur.round;
                        if (round && ok) ok = __all_sync(0xffffffffu, wait(&sm.empty[st], (round - 1) & 1, sm, a.b.guard));
                        if (kv == 0) {
                            // The slot of this unit's scales is free: with at most 6 stages the V tile stored last took
                            // the place of one whose P V had completed, of the unit kScaleUnits back or a later one.
                            const unsigned slot = unit % kScaleUnits;
                            // The largest v scale of the unit, over the four warps.
                            float top = warp_max(vs);
                            float* red = reinterpret_cast<float*>(&sm) + (kHead - 64) / 4 + 4 * (unit & 1);
                            if (lane == 0) red[warp & 3] = top;
                            stop = !feeders_agree(ok);
                            if (stop) break;
                            top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
                            g = max(g, ceil_log2(top));
                            const uint32_t at = scales + slot * (2 * kUnit * 4) + 4 * e0;
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(ks) : "memory");
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * kUnit), "f"(vs * pow2i(-g)) : "memory");
                            if (e0 == 0) {
                                sm.g[slot] = g;
                                sm.bad[unit & 7] = (bad & 0xffu);
                            }
                        }
                        if (!ok) break;     // the others learn of it at the next unit's barrier
                        const uint32_t tile = ring + st * kTileBytes;
#pragma unroll
                        for (int i = 0; i < kPieces; ++i) {
                            uint32_t o[8];
                            widen16<K, BF16>(raw[i], o);
                            const int r = row0 + 32 * (i & 3);
                            const uint32_t at = tile + (i >> 2) * kHalfBytes + r * 128;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                                 at + (((2 * piece + j) ^ (r & 7)) << 4)),
                                             "r"(o[4 * j]), "r"(o[4 * j + 1]), "r"(o[4 * j + 2]), "r"(o[4 * j + 3])
                                             : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.full[st]);
                        cur.next(args.stages);
                    }
                    if (stop) break;
                }
                next_tile<kUnit, kCost>(a, work, t);
                if (t.n <= 0) break;
            }
        }
    }
    if (tid == 0 && !open) a.parts.info[blockIdx.x].n = 0;
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, kTmemCols);
    // The few-rows kernel before this one may still run: whoever waits for this
    // kernel waits for both.
    pdl_wait();
}

// A pool's tensor map: 64 dims of `box` positions of one head and page per
// copy.  The dims stand in the order of their strides, rank[] says where
// position, head and page went.
bool encode_pool(CUtensorMap* m, const char* base, const Pool& kv, int head_dim, bool bf16, int (&rank)[3]) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int page = 1 << kv.page_shift;
    long long stride[3] = {kv.token_bytes, kv.head_bytes, kv.page_bytes};
    const unsigned long long size[3] = {(unsigned long long)page, (unsigned long long)kv.n_kv,
                                        (unsigned long long)kv.n_pages};
    // A dim of one element may have any stride.
    for (int i = 0; i < 3; ++i)
        if (size[i] == 1) stride[i] = (long long)head_dim * 2 << 20;
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (stride[order[j]] > stride[order[j + 1]]) {
                const int x = order[j];
                order[j] = order[j + 1];
                order[j + 1] = x;
            }
    cuuint64_t dims[4] = {(cuuint64_t)head_dim, 1, 1, 1}, strides[3];
    cuuint32_t box[4] = {64, 1, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        const int d = order[i];
        rank[d] = i;
        dims[1 + i] = size[d];
        strides[i] = (cuuint64_t)stride[d];
        if (d == 0) box[1 + i] = (cuuint32_t)(page < kUnit ? page : kUnit);
    }
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<char*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_q(CUtensorMap* m, const Rows& q, int n_rows, int n_head, int group, int sub_rows, int head_dim, bool bf16) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)n_head, (cuuint64_t)n_rows};
    const cuuint64_t strides[2] = {n_head > 1 ? (cuuint64_t)q.head_bytes : (cuuint64_t)head_dim * 2,
                                   n_rows > 1 ? (cuuint64_t)q.row_bytes : (cuuint64_t)head_dim * 2 * n_head};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)sub_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, q.data, dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool BF16, Kind K>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, TcArgs& args, int n_sm,
                   bool chained, cudaStream_t st) {
    constexpr int kTileBytes = HD / 64 * kHalfBytes, kThreads = Split<K>::kThreads;
    auto kern = k_paged_attn_tc<HD, BF16, K>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    const int rest = kStaging + 8 * (args.a.b.n_seq + 1) + (K == kSame16 ? 0 : kScaleUnits * 2 * kUnit * 4);
    const int room = 227 * 1024 - 1024 - kHead - rest - 2 * kTileBytes;
    args.stages = min(K == kSame16 ? kMaxStages : kMaxStages8, room / kTileBytes);
    const size_t smem = 1024 + kHead + (size_t)(2 + args.stages) * kTileBytes + rest;
    if (chained) return launch_pdl(kern, dim3(n_sm), dim3(kThreads), smem, st, q, k, v, args);
    kern<<<n_sm, kThreads, smem, st>>>(q, k, v, args);
    return cudaGetLastError();
}

template <Kind K>
cudaError_t launch_hd(const TcMaps& m, TcArgs& args, int head_dim, bool bf16, int n_sm, bool chained, cudaStream_t st) {
    if (head_dim == 64)
        return bf16 ? launch<64, true, K>(m.q, m.k, m.v, args, n_sm, chained, st)
                    : launch<64, false, K>(m.q, m.k, m.v, args, n_sm, chained, st);
    return bf16 ? launch<128, true, K>(m.q, m.k, m.v, args, n_sm, chained, st)
                : launch<128, false, K>(m.q, m.k, m.v, args, n_sm, chained, st);
}

}  // namespace

int tc_tile_rows(int group) { return 2 * (128 / group) * group; }

bool tc_encode(TcMaps& m, const Pool& kv, const AttnCall& c, const Rows& q, int n_rows) {
    const bool bf16 = c.dtype == QWEN2_DTYPE_BF16;
    const int group = c.n_head / kv.n_kv;
    int rank_v[3];
    if (!encode_q(&m.q, q, n_rows, c.n_head, group, 128 / group, c.head_dim, bf16)) return false;
    if (c.format == QWEN2_KV_INT8 || c.format == QWEN2_KV_E4M3) {
        m.k = m.v = m.q;      // not used
        return true;
    }
    return encode_pool(&m.k, kv.k, kv, c.head_dim, bf16, m.kv_rank) &&
           encode_pool(&m.v, kv.v, kv, c.head_dim, bf16, rank_v);
}

cudaError_t enqueue_attention_tc(const TcMaps& m, const AttnArgs& a, int format, int head_dim, bool bf16, int n_sm,
                                 bool chained, cudaStream_t st) {
    TcArgs args{};
    args.a = a;
    args.sub = a.tile / 2;
    args.sub_rows = args.sub / a.group;
    for (int i = 0; i < 3; ++i) args.kv_rank[i] = m.kv_rank[i];
    args.min_slots = kCost + 2;
    if (format == QWEN2_KV_INT8) return launch_hd<kInt8>(m, args, head_dim, bf16, n_sm, chained, st);
    if (format == QWEN2_KV_E4M3) return launch_hd<kE4m3>(m, args, head_dim, bf16, n_sm, chained, st);
    return launch_hd<kSame16>(m, args, head_dim, bf16, n_sm, chained, st);
}

}  // namespace paged
}  // namespace qwen2
