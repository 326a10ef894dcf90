// Shared by the paged key / value cache operators: the descriptors as the
// kernels take them, sequence and page lookups with their bounds checks, and
// the work list of the attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qwen2.h"
#include "common.cuh"

namespace qwen2 {
namespace paged {

// The pool and the batch, checked on the host (paged_api.cu).
struct Pool {
    char *k, *v;
    float *k_scale, *v_scale;
    int n_pages, page_shift;                            // page_size = 1 << page_shift
    int n_kv;
    long long page_bytes, token_bytes, head_bytes;      // strides in bytes
};
struct Batch {
    int n_seq, n_rows, max_q, max_pages;
    long long pages_stride;
    const int *q_start, *kv_len, *pages;
    int* guard;
};
struct Rows {
    char* data;
    long long row_bytes, head_bytes;                    // strides in bytes
};

// One sequence's rows [q0, q0 + n) and positions [0, kv), clamped to what the
// buffers hold, so that bad device values never lead outside them.
struct Seq {
    int q0, n, kv;
    bool bad_rows, bad_len;
};
__device__ __forceinline__ Seq load_seq(const Batch& b, int page_shift, int s) {
    Seq r;
    const int q0 = b.q_start[s], q1 = b.q_start[s + 1], kv = b.kv_len[s];
    r.bad_rows = q0 < 0 || q1 < q0 || q1 > b.n_rows || q1 - q0 > b.max_q;
    r.q0 = min(max(q0, 0), b.n_rows);
    r.n = r.bad_rows ? 0 : q1 - q0;
    const long long cap = (long long)b.max_pages << page_shift;
    r.bad_len = kv < 0 || kv > cap;
    r.kv = r.bad_len ? 0 : kv;
    return r;
}

// ---- the attention kernels' work list -------------------------------------------
// The query rows of one sequence and kv head are the pairs (row, query head of
// the group), row-major: packed row i = row * group + head.  They are cut into
// tiles of `tile` packed rows, and each tile's keys into units of kKeys
// positions; a tile without keys is one unit.  Every tile takes kCost slots
// for what it costs beside its units (its queries, its rows on their way out)
// and one per unit; the slots of all tiles, ordered (sequence, kv head, tile,
// unit), form one list, of which CTA c of g takes the contiguous c-th part:
// every CTA has the same work whatever the mix of lengths, and a tile is cut
// at most where two CTAs' parts meet (a cut among the kCost slots leaves the
// tile to the later CTA).  A CTA that covers a whole tile writes its rows
// itself; the others leave a partial (row maxima, sums, unnormalised rows)
// that k_attn_join adds up in list order, so results do not depend on timing.

// Keys that the tile of packed rows [i0, i0 + rows) sees: its last row's.
__device__ __forceinline__ int tile_keys(const Seq& q, int group, int i0, int rows, bool causal) {
    if (!causal) return q.kv;
    const int last = (min(i0 + rows, q.n * group) - 1) / group;
    return max(0, q.kv - q.n + last + 1);
}
// Units of one tile.
template <int kKeys>
__device__ __forceinline__ int tile_units(const Seq& q, int group, int t, int rows, bool causal) {
    return max(1, (tile_keys(q, group, t * rows, rows, causal) + kKeys - 1) / kKeys);
}

// What a CTA left in the workspace: slot 0 the part of a tile that an earlier
// CTA began, slot 1 the beginning of a tile that goes on in the next CTAs;
// PartInfo describes slot 1.
struct PartInfo {
    int n;                               // parts of the tile, this one included; 0: no open tile
    int q0, packed0, packed_end, head;   // rows of the batch from q0; packed rows [packed0, packed_end) of kv head `head`
    int pad[3];
};

// The workspace of one attention kernel: g CTAs of tiles of `rows` packed rows.
struct Parts {
    PartInfo* info;   // [g]
    float* ml;        // [2 g][2][rows]: row maxima (base 2), sums
    float* o;         // [2 g][rows][hd], or (beside) [2 g][hd / 4][rows][4]
    int rows;
    bool beside;      // rows side by side, four dims each
};
__host__ __device__ inline long long parts_bytes(int g, int rows, int hd) {
    const long long b = (long long)g * (sizeof(PartInfo) + 2 * (2ll * rows * 4 + (long long)rows * hd * 4));
    return (b + 255) / 256 * 256;
}
inline Parts carve_parts(void* ws, int g, int rows, bool beside) {
    Parts p;
    char* c = static_cast<char*>(ws);
    p.info = reinterpret_cast<PartInfo*>(c);
    p.ml = reinterpret_cast<float*>(c + (long long)g * sizeof(PartInfo));
    p.o = p.ml + 4ll * g * rows;
    p.rows = rows;
    p.beside = beside;
    return p;
}

// Everything an attention kernel takes.
struct AttnArgs {
    Pool kv;
    Batch b;
    Rows q, out;
    float* lse;              // [n_rows][n_head] or null
    int n_head, group;
    int causal;
    float scale_log2;        // scale * log2(e): the softmax runs in base 2
    int rows_lo, rows_hi;    // this kernel's sequences: rows_lo < packed rows <= rows_hi
    int tile;                // packed rows per tile
    Parts parts;
};

// One CTA's current tile.
struct Tile {
    int s, head, t;          // sequence, kv head, tile index
    Seq q;
    int keys, units;         // keys the tile sees, and their units
    long long at;            // its first slot in the list
    int u0, n;               // first unit and number of units of this CTA's part; n <= 0: past its end
};

// a / b of non-negative numbers; a division of 64 bits is some 100 dependent
// instructions, and the work list's numbers rarely need one (a call, to keep
// it out of the kernels' instruction cache lines).
static __device__ __noinline__ long long div_long(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long div_pos(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return div_long(a, b);
}

// Slots of one kv head of the first s sequences, and the CTA's share.
struct WorkList {
    const long long* prefix;   // shared memory [n_seq + 1]
    long long begin, end;      // this CTA's slots
    long long each, rest;      // the first `rest` CTAs take each + 1 slots, the others `each`
    __device__ __forceinline__ int owner(long long slot) const {
        const long long big = rest * (each + 1);
        return (int)(slot < big ? div_pos(slot, each + 1) : rest + div_pos(slot - big, each));
    }
};

__device__ __forceinline__ bool owns(const AttnArgs& a, const Seq& q) {
    const long long packed = (long long)q.n * a.group;
    return packed > a.rows_lo && packed <= a.rows_hi;
}

// Builds the prefix sums with the whole block (at most 4096 sequences and 32
// warps, at least 4) and returns this CTA's share.  A CTA gets at least
// kMin > kCost slots, so that small batches are not cut finer than pays and
// every part has a unit.  A warp takes 32 sequences at a time; up to 32 need a
// single barrier.
template <int kKeys, int kCost, int kMin>
__device__ __forceinline__ WorkList build_work(const AttnArgs& a, long long* prefix) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll 1
    for (int s0 = 32 * warp; s0 < a.b.n_seq; s0 += 32 * warps) {
        const int s = s0 + lane;
        long long u = 0;
        Seq q{};
        bool many = false;
        if (s < a.b.n_seq) {
            q = load_seq(a.b, a.kv.page_shift, s);
            if (blockIdx.x == 0 && (q.bad_rows || q.bad_len))
                raise_guard(a.b.guard, q.bad_rows ? kGuardShape : kGuardPosition);
            if (owns(a, q)) {
                const int tiles = (q.n * a.group + a.tile - 1) / a.tile;
                many = a.causal && tiles > 1;
                u = (long long)tiles * (kCost + tile_units<kKeys>(q, a.group, 0, a.tile, a.causal));
            }
        }
        // Causal tiles each have a length of their own: the whole warp counts them.
        for (unsigned left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
            const int src = __ffs(left) - 1;
            Seq w{};
            w.n = __shfl_sync(0xffffffffu, q.n, src);
            w.kv = __shfl_sync(0xffffffffu, q.kv, src);
            const int tiles = (w.n * a.group + a.tile - 1) / a.tile;
            long long sum = 0;
            for (int t = lane; t < tiles; t += 32) sum += kCost + tile_units<kKeys>(w, a.group, t, a.tile, true);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == src) u = sum;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) u += v;
        }
        if (s < a.b.n_seq) prefix[s + 1] = u;
    }
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (a.b.n_seq > 32) {
        // Each 32's sums are their own so far: lane k holds what comes before
        // the warp's k-th 32.
        long long before = 0;
        int k = 0;
        for (int s0 = 32 * warp; s0 < a.b.n_seq; s0 += 32 * warps, ++k) {
            long long sum = 0;
            for (int c = 32 * (lane + 1); c <= s0; c += 1024) sum += prefix[c];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == k) before = sum;
        }
        __syncthreads();
        k = 0;
        for (int s0 = 32 * warp; s0 < a.b.n_seq; s0 += 32 * warps, ++k) {
            const long long add = __shfl_sync(0xffffffffu, before, k);
            if (s0 + lane < a.b.n_seq) prefix[s0 + lane + 1] += add;
        }
        __syncthreads();
    }
    const long long total = prefix[a.b.n_seq] * a.kv.n_kv;
    const long long most = (long long)((unsigned long long)total / kMin);
    const long long g = most < (long long)gridDim.x ? (most > 0 ? most : 1) : (long long)gridDim.x;
    WorkList w;
    w.prefix = prefix;
    const long long c = blockIdx.x;
    // total / g and the remainder keep the products within 64 bits.
    w.each = div_pos(total, g);
    w.rest = total - w.each * g;
    w.begin = c < g ? w.each * c + (c < w.rest ? c : w.rest) : total;
    w.end = c < g ? w.begin + w.each + (c < w.rest ? 1 : 0) : total;
    return w;
}

// The CTA's part of a tile whose `at` and `units` are set.
template <int kCost>
__device__ __forceinline__ void set_part(const WorkList& w, Tile& t) {
    t.u0 = (int)max(0ll, w.begin - t.at - kCost);
    t.n = (int)min((long long)t.units, max(0ll, w.end - t.at - kCost)) - t.u0;
}

// The tile that holds the CTA's first slot.  Called by whole warps, for a part
// that is not empty.
template <int kKeys, int kCost>
__device__ __forceinline__ Tile find_tile(const AttnArgs& a, const WorkList& w) {
    int lo = 0, hi = a.b.n_seq;          // the largest s that begins at or before it has slots of its own
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (w.prefix[mid] * a.kv.n_kv <= w.begin) lo = mid;
        else hi = mid;
    }
    Tile t;
    t.s = lo;
    t.q = load_seq(a.b, a.kv.page_shift, lo);
    const long long per_head = w.prefix[lo + 1] - w.prefix[lo];
    long long r = w.begin - w.prefix[lo] * a.kv.n_kv;
    t.head = (int)div_pos(r, per_head);
    r -= t.head * per_head;
    const int tiles = (t.q.n * a.group + a.tile - 1) / a.tile;
    if (!a.causal) {
        const int slots = kCost + tile_units<kKeys>(t.q, a.group, 0, a.tile, false);
        t.t = (int)div_pos(r, slots);
        r -= (long long)t.t * slots;
    } else {
        // 32 tiles at a time: the first one whose slots reach past r.
        const int lane = threadIdx.x & 31;
        for (int t0 = 0;; t0 += 32) {
            const int own = t0 + lane < tiles ? kCost + tile_units<kKeys>(t.q, a.group, t0 + lane, a.tile, true) : 0;
            long long sum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, sum > r);
            const int at = hit ? __ffs(hit) - 1 : 31;
            const long long before = __shfl_sync(0xffffffffu, sum - own, at);
            t.t = t0 + at;
            if (hit || t0 + 32 >= tiles) {
                r -= before;
                break;
            }
            r -= __shfl_sync(0xffffffffu, sum, 31);
        }
        t.t = min(t.t, tiles - 1);
    }
    t.keys = tile_keys(t.q, a.group, t.t * a.tile, a.tile, a.causal);
    t.units = max(1, (t.keys + kKeys - 1) / kKeys);
    t.at = w.begin - r;
    set_part<kCost>(w, t);
    return t;
}

// The tile after `t` in the list; its n is <= 0 past the CTA's part.
template <int kKeys, int kCost>
__device__ __forceinline__ void next_tile(const AttnArgs& a, const WorkList& w, Tile& t) {
    t.at += kCost + t.units;
    t.n = 0;
    if (t.at + kCost >= w.end) return;
    const int tiles = (t.q.n * a.group + a.tile - 1) / a.tile;
    if (++t.t >= tiles) {
        t.t = 0;
        if (++t.head == a.kv.n_kv) {
            t.head = 0;
            do ++t.s;
            while (t.s + 1 < a.b.n_seq && w.prefix[t.s + 1] == w.prefix[t.s]);
            if (t.s >= a.b.n_seq) return;
            t.q = load_seq(a.b, a.kv.page_shift, t.s);
        }
    }
    t.keys = tile_keys(t.q, a.group, t.t * a.tile, a.tile, a.causal);
    t.units = max(1, (t.keys + kKeys - 1) / kKeys);
    set_part<kCost>(w, t);
}

// How a CTA's part of a tile lies in it, and where its partial goes.
struct PartPlace {
    bool whole, begins;
    int slot;
};
__device__ __forceinline__ PartPlace part_place(const Tile& t) {
    PartPlace p;
    p.begins = t.u0 == 0;
    p.whole = p.begins && t.n >= t.units;
    p.slot = 2 * blockIdx.x + (p.begins ? 1 : 0);
    return p;
}
// By one thread, for a tile that begins here and goes on in the next CTA.
template <int kCost>
__device__ __forceinline__ void note_open(const AttnArgs& a, const WorkList& w, const Tile& t) {
    PartInfo pi;
    pi.n = w.owner(t.at + kCost + t.units - 1) - (int)blockIdx.x + 1;
    pi.q0 = t.q.q0;
    pi.packed0 = t.t * a.tile;
    pi.packed_end = min(pi.packed0 + a.tile, t.q.n * a.group);
    pi.head = t.head;
    a.parts.info[blockIdx.x] = pi;
}

// Last position packed row i of a sequence sees.
__device__ __forceinline__ int row_limit(const AttnArgs& a, const Seq& q, int i) {
    return a.causal ? q.kv - q.n + i / a.group : q.kv - 1;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace paged
}  // namespace qwen2
