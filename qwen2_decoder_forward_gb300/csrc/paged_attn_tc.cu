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
// 64 positions and half:  S = Q K^T into 64 columns of TMEM; thread i of the
// half's warpgroup owns row i, takes S into registers, writes P = 2^(s - m)
// as 16-bit pairs back over S, and the tensor core takes P from there:
// O += P V.
//
// Each half has two S buffers: S of the next unit is there when a softmax
// ends, and the softmaxes run back to back while the products of the unit
// before and of the unit after next are made; S of a unit is issued once P V
// of the unit two before, which used its buffer, has completed.  (One buffer
// of 128 positions, with S behind P V, left the tensor pipe idle half the
// time: softmax, P V, S and three hand-overs of 200 to 300 cycles in a row.)
//
// Warps: 0-3 softmax of A, 4-7 of B; 8 issues S of both (and asks for the
// queries), 9 P V of both; 10 loads pages.  S and P V have a thread each, since
// S of a unit waits for P V of an earlier one and every wait or commit costs
// the issuing thread 100 to 150 cycles (one thread for all of a half's products
// took 2,160 cycles a unit, half of them waits).  TMEM (512 columns): S at
// 128 x + 64 b for buffer b of half x, O from 256.
//
// 8-bit pages: TMA brings codes and scales into a ring of their own, and four
// more warps (12-15) widen the codes to exact 16-bit values (of the queries'
// type) in the swizzled tiles that TMA would have written (loading them
// through registers ran at a third of the speed: a page id, codes and scales
// in flight share a warp's few load counters, and each wait for one was a wait
// for all).  The scales stay out of the products: k's multiplies the scores,
// v's the probabilities, relative to G, the largest v scale so far rounded up
// to a power of two, which O carries like the reference m.
//
// Measured: a prompt of 5,001 rows (28 heads on 4 of 128, bf16) 200 us, 895
// TFLOP/s, the join's 15 us included; 1,024 rows after 31,000 positions of e4m3
// 604 us, 766 TFLOP/s.  A unit takes some 1,930 cycles, as long as its products
// take one after another (16 of S at 79 cycles each, 8 of P V at 86), S at half
// the pipe's rate, since an M = 128 product of N = 64 takes as long as one of
// N = 128 (the counters show the pipe busy 64% of the time).  Beside: 3,000 to
// 8,000 cycles where a CTA changes tiles (the last softmaxes, rows out through
// shared memory, new queries), and about 9,000 before its first product, which
// with the join is most of a short chunk's time.
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

constexpr int kUnit = 64;                  // positions per unit
constexpr int kCost = 4;                   // slots of a tile beside its units (paged.cuh)
enum Kind { kSame16, kInt8, kE4m3 };
constexpr int kFeeders = 4;                // warps that widen 8-bit codes
template <Kind K>
constexpr int kThreadsOf = K == kSame16 ? 352 : 512;
constexpr int kStaging = 8 * 2048;         // output rows on their way, 2 KB per softmax warp
constexpr int kLag = 8;                    // units whose scales are kept
constexpr int kBadLag = 16;                // units whose bad pages are kept: they are noted earlier
constexpr int kMaxStages = 6;              // K tiles, and V tiles, in the ring.  At most kLag - 2, so that the slot
                                           // of a unit's scales is free when its K is stored: the V stored just
                                           // before, of the unit two back, took the place of one whose P V had
                                           // completed.
constexpr int kTiles8 = 3;                 // 8-bit pages: K tiles, and V tiles
constexpr int kMaxRaw = 6;                 // 8-bit pages: tiles of codes; kMaxRaw / 2 + 2 + kTiles8 <= kBadLag
constexpr int kRawScales = 2 * kUnit * 4;  // k's and v's scales behind each tile of codes
constexpr int kQBytes = 128 * 128;         // 128 rows of 64 16-bit elements
constexpr int kHalfBytes = kUnit * 128;    // 64 positions of 64 16-bit elements
constexpr uint32_t kTmemCols = 512;
constexpr float kSlack = 8.f;              // log2 of the growth that is left in the weights

// s_full, p_full and o_full have a barrier per buffer: unit n of a half is
// phase n / 2 of barrier n % 2.  Up to two units are under way at once, and a
// parity wait can tell only the current phase from the one before it.
struct TcSmem {
    uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
    uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], o_full[2][2], tail, drain[2];
    unsigned bad[kBadLag];                 // per unit (mod kBadLag): its positions in bad pages, 16 per bit
    int g[kLag];                           // 8-bit pages, per unit: log2 of G
    uint32_t tmem_slot;
    int abort;
};
constexpr int kHead = 1024;                // TcSmem, in front of the 1024-byte aligned tiles
static_assert(sizeof(TcSmem) <= kHead, "");

struct TcArgs {
    AttnArgs a;
    int sub;              // packed rows of a half: R * group
    int sub_rows;         // R
    int k_stages, v_stages, raw_stages;
    int kv_rank[3];       // tensor-map dims (1..3) of position, head, page
};

// The roles' loops together have to stay within the instruction cache (inlined
// everywhere, the slow part of the waits and the walk over the work list made
// instruction fetches the largest stall of the 8-bit kernels): those are calls.
// The 8-bit kernels, with one role more, call for their first tile as well:
// 1,024 rows after 31,000 positions of e4m3 take 606 us so and 661 us without;
// the others are quicker on their way to it without the call (a call reads the
// kernel's parameters from memory): a batch of short chunks 31.5 against 32.7 us.
__device__ __noinline__ Tile tc_find_tile(const AttnArgs& a, const WorkList& w) { return find_tile<kUnit, kCost>(a, w); }
template <bool kCall>
__device__ __forceinline__ Tile first_tile(const AttnArgs& a, const WorkList& w) {
    if constexpr (kCall) return tc_find_tile(a, w);
    else return find_tile<kUnit, kCost>(a, w);
}
__device__ __noinline__ void tc_next_tile(const AttnArgs& a, const WorkList& w, Tile& t) {
    next_tile<kUnit, kCost>(a, w, t);
}
__device__ __noinline__ void tc_note_open(const AttnArgs& a, const WorkList& w, const Tile& t) {
    note_open<kCost>(a, w, t);
}

// Waits for the phase of parity `parity`, at most about kWaitNs: the SM's own
// clock is read (a read of the global timer costs a large part of a unit's
// time).  False once this or another wait of the block has given up.
constexpr long long kWaitClocks = (long long)kWaitNs * 2;      // 2 s or more at up to 2 GHz
__device__ __noinline__ bool wait_slow(uint64_t* bar, unsigned parity, TcSmem& sm, int* guard) {
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
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

// Untiled copy of `bytes` (a multiple of 16, both ends 16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, int bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A place in the ring of K tiles or of V tiles: stored and used in order.
struct Cursor {
    int stage = 0;
    unsigned round = 0;
    __device__ __forceinline__ void next(int stages) {
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
    static constexpr uint32_t s(int x, int b) { return 128u * x + 64u * b; }
    static constexpr uint32_t o(int x) { return 256u + (uint32_t)HD * x; }
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

// The i-th of the 2 n tiles of n units in the order they are loaded, K of a
// unit before V of the one before it (K0 K1 V0 K2 V1 ... V of the last): 0 for
// K, 1 for V of unit u.  The loops over it have one copy of their body: the
// warps' roles together have to stay within the instruction cache (three
// copies of the widening loop made fetches the largest stall by far).
__device__ __forceinline__ int in_order(int i, int n, int& u) {
    const bool last = i == 2 * n - 1, v = last || (i > 0 && !(i & 1));
    u = last ? n - 1 : v ? i / 2 - 1 : (i + 1) / 2;
    return v;
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

template <int HD, bool BF16, Kind K>
__global__ void __launch_bounds__(kThreadsOf<K>, 1)
    k_paged_attn_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcArgs args) {
    using T = Tmem<HD>;
    constexpr int kHalves = HD / 64;
    constexpr int kQTile = kHalves * kQBytes, kTile = kHalves * kHalfBytes;
    constexpr bool k8 = K != kSame16;
    const AttnArgs& a = args.a;
    extern __shared__ unsigned char tc_smem_raw[];
    const uint32_t pad = (1024u - (smem_addr(tc_smem_raw) & 1023u)) & 1023u;
    TcSmem& sm = *reinterpret_cast<TcSmem*>(tc_smem_raw + pad);
    const uint32_t q_tiles = smem_addr(&sm) + kHead;                 // A, B
    const uint32_t k_ring = q_tiles + 2 * kQTile, v_ring = k_ring + args.k_stages * kTile;
    const uint32_t staging = v_ring + args.v_stages * kTile;
    // 8-bit pages: tiles of codes [64-dim half][kUnit][64 bytes] and their scales, then [kLag][k, v / G][kUnit] f32.
    constexpr int kRaw = kHalves * kUnit * 64 + kRawScales;
    const uint32_t raw_ring = staging + kStaging, scales = raw_ring + args.raw_stages * kRaw;
    long long* prefix = reinterpret_cast<long long*>(tc_smem_raw + pad + kHead + 2 * kQTile +
                                                     (args.k_stages + args.v_stages) * kTile + kStaging +
                                                     (k8 ? args.raw_stages * kRaw + kLag * 2 * kUnit * 4 : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_launch_dependents();
    if (tid == 9 * 32) {
#pragma unroll 1
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sm.k_full[i], k8 ? kFeeders : 1);
            mbar_init(&sm.v_full[i], k8 ? kFeeders : 1);
            mbar_init(&sm.k_empty[i], 2);
            mbar_init(&sm.v_empty[i], 2);
        }
#pragma unroll 1
        for (int i = 0; i < kMaxRaw; ++i) {
            mbar_init(&sm.raw_full[i], 1);
            mbar_init(&sm.raw_empty[i], kFeeders);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sm.s_full[x][0], 1);
            mbar_init(&sm.s_full[x][1], 1);
            mbar_init(&sm.p_full[x][0], 128);
            mbar_init(&sm.p_full[x][1], 128);
            mbar_init(&sm.o_full[x][0], 1);
            mbar_init(&sm.o_full[x][1], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&sm.drain[i], 1);
        mbar_init(&sm.tail, 1);
        mbar_init_fence();
        sm.abort = 0;
    }
    if (warp == 8) tmem_alloc(&sm.tmem_slot, kTmemCols);
    if (warp == 10 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    const WorkList work = build_work<kUnit, kCost, kCost + 4>(a, prefix);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_slot;
    bool open = false;
    if (work.begin < work.end) {
        Tile t = first_tile<k8>(a, work);
        if (warp < 8) {
            // ---- softmax of half x --------------------------------------------------
            const int x = warp >> 2, rl = 32 * (warp & 3) + lane;
            const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            const uint32_t t_o = lanes + T::o(x);
            const float sc = a.scale_log2;
            unsigned n_s = 0;          // units of this half so far
            unsigned unit = 0;         // units of the CTA before this tile
            Cursor ck, cv;             // K of the current unit; V of the oldest unit not yet released
            bool ok = true;
#pragma unroll 1
            while (ok) {
                const int packed0 = t.t * a.tile, packed = t.q.n * a.group;
                const int i = packed0 + x * args.sub + rl;
                const bool live = rl < args.sub && i < packed;
                if (packed0 + x * args.sub < packed) {
                    const int lim = live ? min(row_limit(a, t.q, i), t.keys - 1) : t.keys - 1;
                    const int sure = min(row_limit(a, t.q, packed0 + x * args.sub), t.keys - 1);
                    float m = -INFINITY, l0 = 0.f, l1 = 0.f;
                    int g = -100;          // log2 of G
#pragma unroll 1
                    for (int u = 0; u < t.n; ++u, ++n_s) {
                        const int key0 = (t.u0 + u) * kUnit;
                        const uint32_t t_s = lanes + T::s(x, n_s & 1);
                        ok = __all_sync(0xffffffffu, wait(&sm.s_full[x][n_s & 1], n_s >> 1 & 1, sm, a.b.guard));
                        if (!ok) break;
                        tc_fence_after();
                        uint32_t s[2][32];
                        tmem_ld32_async(t_s, s[0]);
                        tmem_ld32_async(t_s + 32, s[1]);
                        const unsigned slot = (unit + u) % kLag;
                        const unsigned bad = sm.bad[(unit + u) % kBadLag];
                        if (rl == 0) {
                            // This half is done with the unit's K tile, with the queries after the
                            // last one, and (S was issued after that P V had completed) with V of
                            // the unit two before.
                            mbar_arrive(&sm.k_empty[ck.stage]);
                            if (u + 1 == t.n) mbar_arrive(&sm.q_empty);
                            if (u > 1) mbar_arrive(&sm.v_empty[cv.stage]);
                        }
                        ck.next(args.k_stages);
                        if (u > 1) cv.next(args.v_stages);
                        const uint32_t at = scales + slot * (2 * kUnit * 4);
                        tmem_ld_wait();
                        pin32(s[0]);
                        pin32(s[1]);
                        if constexpr (k8) {
                            scale_scores(s[0], at);
                            scale_scores(s[1], at + 128);
                        }
                        if (key0 + kUnit - 1 > sure || bad) {
                            // A bit for each position that the row sees.
                            const int last = lim - key0;
                            unsigned long long see = last >= kUnit - 1 ? ~0ull : last < 0 ? 0ull : (2ull << last) - 1;
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (bad >> c & 1) see &= ~(0xffffull << (16 * c));
                            const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                if (!(lo >> e & 1)) s[0][e] = 0xff800000u;
                                if (!(hi >> e & 1)) s[1][e] = 0xff800000u;
                            }
                        }
                        float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                v[e / 2 & 3] = max3(v[e / 2 & 3], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                        const float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) * sc;
                        // A new reference once the maximum has outgrown the old one.
                        const bool move = top > m + kSlack;
                        float corr = 1.f;
                        if (move) {
                            corr = ex2(m - top);
                            m = top;
                            l0 *= corr;
                            l1 *= corr;
                        }
                        bool scale_o = __any_sync(0xffffffffu, move);
                        if constexpr (k8) {
                            const int ng = sm.g[slot];
                            corr *= pow2i(max(g - ng, -126));
                            scale_o = scale_o || ng != g;
                            g = ng;
                        }
                        if (u > 0 && scale_o) {
                            // P V of the unit before has to be in O (S of this one came after the one
                            // before that).
                            ok = __all_sync(0xffffffffu, wait(&sm.o_full[x][(n_s - 1) & 1], (n_s - 1) >> 1 & 1, sm, a.b.guard));
                            if (!ok) break;
                            tc_fence_after();
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
                            uint32_t p[16];
                            [[maybe_unused]] float4 vs;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float y = __uint_as_float(s[c][2 * e]), z = __uint_as_float(s[c][2 * e + 1]);
                                fma2(y, z, sc, base);
                                y = ex2(y);
                                z = ex2(z);
                                add2(l0, l1, y, z);
                                if constexpr (k8) {
                                    if (e % 2 == 0) vs = lds4(at + 4 * kUnit + 128 * c + 8 * e);
                                    mul2(y, z, e % 2 ? vs.z : vs.x, e % 2 ? vs.w : vs.y);
                                }
                                p[e] = pack2<BF16>(y, z);
                            }
                            tmem_st16(t_s + 16 * c, p);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&sm.p_full[x][n_s & 1]);
                    }
                    if (!ok) break;
                    // ---- the half's rows ------------------------------------------------
                    // The last two P V (S of the last unit came after those before).
                    ok = t.n < 2 || wait(&sm.o_full[x][n_s & 1], (n_s - 2) >> 1 & 1, sm, a.b.guard);
                    ok = __all_sync(0xffffffffu, ok && wait(&sm.o_full[x][(n_s - 1) & 1], (n_s - 1) >> 1 & 1, sm, a.b.guard));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int u = max(0, t.n - 2); u < t.n; ++u) {
                        if (rl == 0) mbar_arrive(&sm.v_empty[cv.stage]);
                        cv.next(args.v_stages);
                    }
                    const float l = l0 + l1, unit_g = k8 ? pow2i(g) : 1.f;
                    const PartPlace place = part_place(t);
                    const int r = x * args.sub + rl;
                    // Finished rows go out through the warp's staging buffer: 64 bytes of each of its 32 rows
                    // at a time, written a row per lane and stored four lanes a row (a row per lane
                    // straight to memory touches 32 lines a store and holds the load / store unit
                    // for 5,000 cycles a tile).  Partials keep four dims of all rows side by side
                    // instead, so that a row per lane is a line (7,500 cycles a tile through the
                    // staging buffer).
                    const float f = !place.whole ? unit_g : l == 0.f ? 0.f : unit_g / l;
                    char* dst = nullptr;
                    float4* part = nullptr;
                    if (place.whole) {
                        const int row = t.q.q0 + i / a.group, qh = t.head * a.group + i % a.group;
                        if (live) dst = a.out.data + (long long)row * a.out.row_bytes + (long long)qh * a.out.head_bytes;
                        if (live && a.lse)
                            a.lse[(long long)row * a.n_head + qh] =
                                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                    } else {
                        part = reinterpret_cast<float4*>(a.parts.o + (long long)place.slot * a.parts.rows * HD) + r;
                        if (live) {
                            a.parts.ml[(long long)place.slot * 2 * a.parts.rows + r] = m;
                            a.parts.ml[((long long)place.slot * 2 + 1) * a.parts.rows + r] = l;
                        }
                    }
                    const uint32_t stage = staging + 2048 * warp;
#pragma unroll 1
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_async(t_o + 32 * c, o);
                        tmem_ld_wait();
                        pin32(o);
                        if (place.whole) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = pack2<BF16>(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
                            put_rows64(stage, w, dst, 64 * c, lane);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (live)
                                    part[(long long)(8 * c + e) * a.parts.rows] = make_float4(
                                        __uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                        __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f);
                        }
                    }
                    if (!place.whole && place.begins) {
                        open = true;
                        if (tid == 0) tc_note_open(a, work, t);
                    }
                    tc_fence_before();
                } else {
#pragma unroll 1
                    for (int u = 0; u < t.n; ++u) {
                        ck.next(args.k_stages);
                        cv.next(args.v_stages);
                    }
                }
                unit += t.n;
                tc_next_tile(a, work, t);
                if (t.n <= 0) break;
            }
        } else if (warp == 8) {
            // ---- queries, and S of both halves ----------------------------------------------
            if (lane == 0) {
                constexpr uint32_t id_s = idesc16(128, kUnit, BF16, false);
                unsigned n[2] = {0, 0}, seg = 0;       // units of each half, tiles
                Cursor ck;
                bool ok = true;
#pragma unroll 1
                for (;; ++seg) {
                    const int halves = t.t * a.tile + args.sub < t.q.n * a.group ? 2 : 1;
                    if (seg) ok = wait(&sm.q_empty, (seg - 1) & 1, sm, a.b.guard);
                    if (!ok) break;
                    mbar_expect_tx(&sm.q_full, (unsigned)(halves * kHalves * args.sub * 128));
                    for (int x = 0; x < halves; ++x)
                        for (int c = 0; c < kHalves; ++c)
                            tma_load_3d(q_tiles + x * kQTile + c * kQBytes, &tm_q, 64 * c, t.head * a.group,
                                        t.q.q0 + (2 * t.t + x) * args.sub_rows, &sm.q_full);
                    ok = wait(&sm.q_full, seg & 1, sm, a.b.guard);
#pragma unroll 1
                    for (int u = 0; u < t.n && ok; ++u) {
                        ok = wait(&sm.k_full[ck.stage], ck.round & 1, sm, a.b.guard);
                        const uint64_t kd = desc_sw128(k_ring + ck.stage * kTile);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (x >= halves) {
                                // No rows in this half: its share of releasing the tile all the same.
                                if (ok) mbar_arrive(&sm.k_empty[ck.stage]);
                                continue;
                            }
                            // The buffer's last P, of the unit two before, has been used.
                            const unsigned b = n[x] & 1;
                            if (n[x] > 1) ok = ok && wait(&sm.o_full[x][b], (n[x] - 2) >> 1 & 1, sm, a.b.guard);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t qd = desc_sw128(q_tiles + x * kQTile);
                            const uint32_t t_s = tmem + T::s(x, b);
#pragma unroll
                            for (int k = 0; k < HD / 16; ++k)
                                mma_f16(t_s, qd + (((k / 4) * kQBytes + (k % 4) * 32) >> 4),
                                        kd + (((k / 4) * kHalfBytes + (k % 4) * 32) >> 4), id_s, k != 0 ? 1u : 0u);
                            mma_commit(&sm.s_full[x][b]);
                            ++n[x];
                        }
                        ck.next(args.k_stages);
                    }
                    if (ok && halves == 1) mbar_arrive(&sm.q_empty);
                    tc_next_tile(a, work, t);
                    if (t.n <= 0 || !ok) break;
                }
                if (!ok) {   // what is in flight ends before the memory is given back
                    mma_commit(&sm.drain[0]);
                    mbar_wait(&sm.drain[0], 0, kWaitNs);
                    mbar_wait(&sm.q_full, seg & 1, kWaitNs);
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---- P V of both halves -----------------------------------------------------------
            if (lane == 0) {
                constexpr uint32_t id_o = idesc16(128, HD, BF16, true);
                unsigned n[2] = {0, 0};
                Cursor cv;
                bool ok = true;
#pragma unroll 1
                while (ok) {
                    const int halves = t.t * a.tile + args.sub < t.q.n * a.group ? 2 : 1;
#pragma unroll 1
                    for (int u = 0; u < t.n && ok; ++u) {
                        ok = wait(&sm.v_full[cv.stage], cv.round & 1, sm, a.b.guard);
                        const uint64_t vd = desc_mn128(v_ring + cv.stage * kTile);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (x >= halves) {
                                if (ok) mbar_arrive(&sm.v_empty[cv.stage]);
                                continue;
                            }
                            const unsigned b = n[x] & 1;
                            ok = ok && wait(&sm.p_full[x][b], n[x] >> 1 & 1, sm, a.b.guard);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int k = 0; k < kUnit / 16; ++k)
                                mma_ts(tmem + T::o(x), tmem + T::s(x, b) + 8 * k, vd + (2048 * k >> 4), id_o,
                                       u > 0 || k > 0 ? 1u : 0u);
                            mma_commit(&sm.o_full[x][b]);
                            ++n[x];
                        }
                        cv.next(args.v_stages);
                    }
                    tc_next_tile(a, work, t);
                    if (t.n <= 0) break;
                }
                if (!ok) {
                    mma_commit(&sm.drain[1]);
                    mbar_wait(&sm.drain[1], 0, kWaitNs);
                }
            }
            __syncwarp();
        } else if (warp == 10) {
            // ---- pages: K of a unit comes a unit before V ----------------------------------------
            const int page_rows = 1 << a.kv.page_shift, box = min(page_rows, kUnit), boxes = kUnit / box;
            constexpr int kRowBytes = k8 ? 64 : 128;     // of a 64-dim half
            const int p = lane / kHalves, h = lane % kHalves;
            unsigned unit = 0, n_tail = 0;
            Cursor ck, cv;                               // 8-bit pages: ck counts the tiles of codes, K and V
            bool ok = true;
            // This lane's page of a unit of the tile, -1 for none (as read: checked when used).
            const auto look_up = [&](int u) {
                const int key = (t.u0 + u) * kUnit + p * box;
                if (u >= t.n || p >= boxes || key >= t.keys) return -1;
                return __ldg(a.b.pages + (long long)t.s * a.b.pages_stride + (key >> a.kv.page_shift));
            };
            // Asks for K (kv = 0) or V of unit u of the tile; `ordinal` is the unit's number in the CTA.
            const auto feed = [&](int u, int kv, int page, unsigned ordinal) {
                Cursor& cur = kv && !k8 ? cv : ck;
                uint64_t* full = k8 ? &sm.raw_full[cur.stage] : kv ? &sm.v_full[cur.stage] : &sm.k_full[cur.stage];
                uint64_t* empty = k8 ? &sm.raw_empty[cur.stage] : kv ? &sm.v_empty[cur.stage] : &sm.k_empty[cur.stage];
                const int key0 = (t.u0 + u) * kUnit, key = key0 + p * box;
                const bool is_bad = p < boxes && key < t.keys && (unsigned)page >= (unsigned)a.kv.n_pages;
                if (is_bad) {
                    page = -1;
                    raise_guard(a.b.guard, QWEN2_GUARD_PAGE);
                }
                const unsigned bad =
                    __reduce_or_sync(0xffffffffu, is_bad ? ((1u << (box / 16)) - 1) << (p * box / 16) : 0u);
                unsigned bytes = (unsigned)(__popc(__ballot_sync(0xffffffffu, page >= 0)) * box * kRowBytes);
                if (k8 && !kv) bytes += bytes / (kHalves * kRowBytes) * 8;               // and their scales
                const bool patch = !k8 && kv && (key0 + kUnit > t.keys || bad);          // positions that are no keys: zeros in V
                if (cur.round) ok = __all_sync(0xffffffffu, wait(empty, (cur.round - 1) & 1, sm, a.b.guard));
                if (!ok) return;
                const int off = key & (page_rows - 1);
                int at[3];
                at[args.kv_rank[0]] = off;
                at[args.kv_rank[1]] = t.head;
                at[args.kv_rank[2]] = page;
                const uint32_t tile = k8 ? raw_ring + cur.stage * kRaw : (kv ? v_ring : k_ring) + cur.stage * kTile;
                uint64_t* bar = patch ? &sm.tail : full;
                if (lane == 0) {
                    if (!kv) sm.bad[ordinal % kBadLag] = bad;
                    mbar_expect_tx(bar, bytes);
                }
                __syncwarp();
                if (page >= 0) {
                    tma_load_4d(tile + (h * kUnit + p * box) * kRowBytes, kv ? &tm_v : &tm_k, 64 * h, at[0], at[1], at[2], bar);
                    if (k8 && !kv && h == 0) {
                        const long long i = (((long long)page * a.kv.n_kv + t.head) << a.kv.page_shift) + off;
                        const uint32_t to = tile + kHalves * kUnit * 64 + 4 * p * box;
                        bulk_load(to, a.kv.k_scale + i, 4 * box, bar);
                        bulk_load(to + 4 * kUnit, a.kv.v_scale + i, 4 * box, bar);
                    }
                }
                cur.next(k8 ? args.raw_stages : kv ? args.v_stages : args.k_stages);
                if (patch) {
                    ok = __all_sync(0xffffffffu, wait(&sm.tail, n_tail & 1, sm, a.b.guard));
                    if (!ok) mbar_wait(&sm.tail, n_tail & 1, kWaitNs);
                    ++n_tail;
                    // Eight lanes a 128-byte row, four rows a store.
#pragma unroll 1
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
                    if (lane == 0) mbar_arrive(full);
                }
            };
#pragma unroll 1
            while (ok) {
                // One copy of the code for K and V (see in_order): pages are looked up two units
                // ahead of K, and kept until V.
                int k0 = look_up(0), k1 = look_up(1), v0 = -1, v1 = -1, held = 0;
#pragma unroll 1
                for (int i = 0; i < 2 * t.n && ok; ++i) {
                    int u;
                    const int kv = in_order(i, t.n, u);
                    const int page = kv ? v0 : k0;
                    if (kv) {
                        v0 = v1;
                        --held;
                    } else {
                        if (held++) v1 = k0;
                        else v0 = k0;
                        k0 = k1;
                        k1 = look_up(u + 2);
                    }
                    feed(u, kv, page, unit + u);
                }
                unit += t.n;
                tc_next_tile(a, work, t);
                if (t.n <= 0) break;
            }
            if (!ok) {   // copies in flight land before the shared memory is given back
                const auto last = [&](uint64_t* full, const Cursor& c, int stages) {   // each stage's last entry
#pragma unroll 1
                    for (int i = 0; i < stages; ++i)
                        if (i < c.stage || c.round) mbar_wait(&full[i], (i < c.stage ? c.round : c.round - 1) & 1, kWaitNs);
                };
                if (k8) last(sm.raw_full, ck, args.raw_stages);
                else {
                    last(sm.k_full, ck, args.k_stages);
                    last(sm.v_full, cv, args.v_stages);
                }
            }
            __syncwarp();
        } else if (k8 && warp >= 12) {
            // ---- codes to tiles ---------------------------------------------------------------------
            // Thread e takes 16-byte piece e % 4 of row e / 4 (+ 32) of each 64-dim half: two adjacent
            // rows' pieces fill all banks, of the codes and of the tiles.
            const int e0 = tid - 384, piece = e0 & 3, row0 = e0 >> 2;
            unsigned unit = 0;
            Cursor cr, ck, cv;
            bool ok = true;
            int g = -100;
            const auto store = [&](int u, int kv, unsigned ordinal) {
                Cursor& cur = kv ? cv : ck;
                ok = wait(&sm.raw_full[cr.stage], cr.round & 1, sm, a.b.guard);
                if (cur.round)
                    ok = ok && wait(kv ? &sm.v_empty[cur.stage] : &sm.k_empty[cur.stage], (cur.round - 1) & 1, sm, a.b.guard);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                const int key0 = (t.u0 + u) * kUnit;
                const unsigned bad = sm.bad[ordinal % kBadLag];
                const uint32_t raw = raw_ring + cr.stage * kRaw;
                const auto is_key = [&](int r) { return key0 + r < t.keys && !(bad >> (r / 16) & 1); };
                if (!kv) {
                    // Every warp has all the unit's v scales, and so the same G.
                    float ks[2], vs[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = lane + 32 * j;
                        const uint32_t from = raw + kHalves * kUnit * 64 + 4 * r;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks[j]) : "r"(from) : "memory");
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs[j]) : "r"(from + 4 * kUnit) : "memory");
                        if (!is_key(r)) ks[j] = vs[j] = 0.f;
                    }
                    g = max(g, ceil_log2(warp_max(fmaxf(vs[0], vs[1]))));
                    if (warp == 12) {
                        const unsigned slot = ordinal % kLag;
                        const float down = pow2i(-g);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t at = scales + slot * (2 * kUnit * 4) + 4 * (lane + 32 * j);
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(ks[j]) : "memory");
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * kUnit), "f"(vs[j] * down) : "memory");
                        }
                        if (lane == 0) sm.g[slot] = g;
                    }
                }
                const uint32_t tile = (kv ? v_ring : k_ring) + cur.stage * kTile;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = row0 + 32 * j;
                    const bool in = is_key(r);
#pragma unroll
                    for (int c = 0; c < kHalves; ++c) {
                        uint4 w;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                     : "r"(raw + (c * kUnit + r) * 64 + 16 * piece)
                                     : "memory");
                        uint32_t o[8];
                        widen16<K, BF16>(in ? w : make_uint4(0, 0, 0, 0), o);
                        const uint32_t at = tile + c * kHalfBytes + r * 128;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             at + (((2 * piece + i) ^ (r & 7)) << 4)),
                                         "r"(o[4 * i]), "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                                         : "memory");
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(kv ? &sm.v_full[cur.stage] : &sm.k_full[cur.stage]);
                    mbar_arrive(&sm.raw_empty[cr.stage]);
                }
                cr.next(args.raw_stages);
                cur.next(kv ? args.v_stages : args.k_stages);
            };
#pragma unroll 1
            while (ok) {
                g = -100;
#pragma unroll 1
                for (int i = 0; i < 2 * t.n && ok; ++i) {
                    int u;
                    const int kv = in_order(i, t.n, u);
                    store(u, kv, unit + u);
                }
                unit += t.n;
                tc_next_tile(a, work, t);
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
bool encode_pool(CUtensorMap* m, const char* base, const Pool& kv, int head_dim, int format, int (&rank)[3]) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int page = 1 << kv.page_shift;
    const bool k8 = format == QWEN2_KV_INT8 || format == QWEN2_KV_E4M3;
    long long stride[3] = {kv.token_bytes, kv.head_bytes, kv.page_bytes};
    const unsigned long long size[3] = {(unsigned long long)page, (unsigned long long)kv.n_kv,
                                        (unsigned long long)kv.n_pages};
    // A dim of one element may have any stride.
    for (int i = 0; i < 3; ++i)
        if (size[i] == 1) stride[i] = (long long)head_dim << 20;
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
    return enc(m, k8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                     : format == QWEN2_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<char*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               k8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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
    constexpr int kQTile = HD / 64 * kQBytes, kTile = HD / 64 * kHalfBytes, kThreads = kThreadsOf<K>;
    auto kern = k_paged_attn_tc<HD, BF16, K>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    constexpr int kRaw = HD * kUnit + kRawScales;
    int rest = kStaging + 8 * (args.a.b.n_seq + 1) + 2 * kQTile;
    const int room = 227 * 1024 - 1024 - kHead;
    if constexpr (K == kSame16) {
        const int tiles = (room - rest) / kTile;
        args.k_stages = min(kMaxStages, tiles / 2);
        args.v_stages = min(kMaxStages, tiles - args.k_stages);
    } else {
        // 4,096 sequences leave room for two K and V tiles at head_dim 128.
        rest += kLag * 2 * kUnit * 4;
        args.k_stages = args.v_stages = room - rest >= 2 * kTiles8 * kTile + 4 * kRaw ? kTiles8 : 2;
        args.raw_stages = min(kMaxRaw, (room - rest - 2 * args.k_stages * kTile) / kRaw);
    }
    const size_t smem = 1024 + kHead + (size_t)(args.k_stages + args.v_stages) * kTile + args.raw_stages * kRaw + rest;
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
    return encode_pool(&m.k, kv.k, kv, c.head_dim, c.format, m.kv_rank) &&
           encode_pool(&m.v, kv.v, kv, c.head_dim, c.format, rank_v);
}

cudaError_t enqueue_attention_tc(const TcMaps& m, const AttnArgs& a, int format, int head_dim, bool bf16, int n_sm,
                                 bool chained, cudaStream_t st) {
    TcArgs args{};
    args.a = a;
    args.sub = a.tile / 2;
    args.sub_rows = args.sub / a.group;
    for (int i = 0; i < 3; ++i) args.kv_rank[i] = m.kv_rank[i];
    if (format == QWEN2_KV_INT8) return launch_hd<kInt8>(m, args, head_dim, bf16, n_sm, chained, st);
    if (format == QWEN2_KV_E4M3) return launch_hd<kE4m3>(m, args, head_dim, bf16, n_sm, chained, st);
    return launch_hd<kSame16>(m, args, head_dim, bf16, n_sm, chained, st);
}

}  // namespace paged
}  // namespace qwen2
