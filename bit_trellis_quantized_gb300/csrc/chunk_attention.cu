// Attention of a chunk of new tokens over a paged key-value cache.
//
// Token t of sequence s stands at position p = lens[s] - (at[s + 1] - at[s]) +
// t - at[s]; per query head, over the keys j <= p of its key head:
//   x_j = scale q . k_j,  m = max_j x_j,  out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
//   lse = m + ln sum_j e^(x_j - m).
//
// A unit is one (sequence, key head, run of tokens); its rows are the pairs of a
// token and a query head of the key head, tokens outermost, in tiles of as many
// whole tokens as 128 rows hold (all 128 where the group of heads divides it). A
// CTA takes a unit, or a run of its keys, in tiles of 128 keys:
//   S = Q K^T (tcgen05, Q and K in shared memory, S in tensor memory), the
//   weights P = 2^(S c - m) by one thread a row, back to tensor memory over S
//   as 16-bit values, O += P V (A from tensor memory, O stays there).
// Warps: 4 a tile of rows for the softmax, 2 that load, one that issues the
// products, one that hands out units. Each runs ahead of the next as far as
// buffers allow, from unit to unit without a barrier of the CTA.
//
//  * Loads: boxes of a page's rows by TMA where pages are multiples of 8 keys
//    (a box takes 128 values of each row: half of the values a box, pages of 16
//    took 773 us where this takes 487, pages of 64 475 and 373; 2048 tokens
//    behind 14336, 2 key heads of 256), other pages row by row with cp.async (744 us). Rows that
//    are not there are zeros and masked.
//  * Rows: O of 128 rows of 256 values and two tiles' S fill tensor memory; with
//    smaller heads two tiles of rows share the keys, and their softmax and
//    products alternate.
//  * Masks: only tiles that not every row sees in full are masked, in tensor
//    memory before the row is read, so that the loop's code is short (unrolled
//    throughout, the code did not fit the instruction cache and took twice the time).
//  * Units: whole ones are taken over one by one by CTAs that are done; where that
//    leaves CTAs idle too long, all units are cut into equal ranges and the parts joined
//    by a second kernel (ca_plan).
//
// The running maximum that P is scaled by is moved, and O multiplied, only
// where a row's maximum rises by more than kTau powers of two over it: with
// the sum scaled alike the result is the same, and O is left alone nearly
// always. Weights enter the second product rounded once to the type (half a
// step of each weight; the sums and lse are of the unrounded ones): two parts
// as in the decode kernel would cost the products half as much again. fp16 ones are
// of the weight times 2^kUp, so that keys at 2^-25 of the largest weight keep
// all but their last bit (steps below 2^-14 are 2^-24); bf16 ones times 2^-kTau, so that none is above 1 and sums of large
// values end as f32 does.
//
// Bound: the products; a tile of 128 rows and keys of 256 values takes 1.37 us,
// 1.86 PFLOP/s (97% of cuBLAS's measured burst), while tiles follow each other. Around them: 6 us a unit, and
// the power limit in long calls. Measured, 16 heads on 2 key heads of 256: 2048
// tokens 36 us (0.96 PFLOP/s), 8192 tokens 390 (1.41), 2048 behind 63488
// 1.52 ms captured (1.42), 1.74 ms in a long run (1.25); 32 heads on 8 of 128, 4096 tokens 121 (1.14).
//
// Running maximum and sum: Milakov and Gimelshein, "Online normalizer calculation
// for softmax", 2018. Tiles of rows in turn, and a maximum that moves only past a
// threshold, are published methods of such kernels as well.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "context.h"
#include "kernels.h"
#include "tcgen05.cuh"
#include "trellis_core.cuh"

#include <type_traits>

namespace escha {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
template <int DT>
constexpr float kTau = DT == 1 ? 4.f : 8.f;  // P is at most 2^(kTau + kUp): 2^15 in fp16, 1 in bf16
template <int DT>
constexpr float kUp = DT == 1 ? 11.f : -kTau<DT>;

constexpr int kKeys = 128;  // of a tile
template <int D>
struct CaCfg {
    static constexpr int kNQ = D == 256 ? 1 : 2;  // tiles of 128 rows: O of both and two S fill tensor memory
    static constexpr int kRows = 128 * kNQ;
    // warps: 4 a tile of rows, then 2 that load, one that issues the products, one that hands out the units
    static constexpr int kSoftWarps = 4 * kNQ, kLoadWarps = 2, kMmaWarp = kSoftWarps + kLoadWarps, kUnitWarp = kMmaWarp + 1;
    static constexpr int kThreads = 32 * (kUnitWarp + 1);
    static constexpr int kSlotD = D < 128 ? D : 128;  // a slot of the ring: 128 keys of up to 128 values
    static constexpr int kParts = D / kSlotD;
    static constexpr int kSlotBytes = kKeys * kSlotD * 2;
    static constexpr int kSlots = D == 64 ? 10 : 5;
    static constexpr int kAhead = D == 64 ? 6 : 3;  // slots whose loads are in flight
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kSmem = kQBytes + kSlots * kSlotBytes + 1024;
    static constexpr uint32_t kScol = 256;  // S of tile q, or of every other tile of keys, at kScol + 128 q
};
constexpr int kMasks = 8;  // (the loads are never more than 5 tiles ahead of the weights)

// n / d of n < 2^31 by one multiplication: mul = ceil(2^(31 + l) / d), l = ceil(log2 d).
struct CaDiv {
    uint32_t mul;
    int shift;
    __device__ __forceinline__ int operator()(int n) const {
        return static_cast<int>((static_cast<unsigned long long>(n) * mul) >> shift);
    }
};

template <int DT>
__device__ __forceinline__ uint32_t ca_pack(float x, float y) {
    if (DT == 1) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sequences' runs of rows, where they are cut over all CTAs, for the join. With the key heads outermost, a unit is (key
// head, run); the places of all units are numbered in this order: a unit has one for each tile of keys, behind kCaStart
// that stand for its beginning and end (queries, first and last products, outputs: about 6 us, with tiles of 1.5).
constexpr int kCaRuns = kSms, kCaStart = 4;
struct CaList {
    int n, places;           // runs, places of all of them
    uint32_t unit[kCaRuns];  // sequence, run << 16
    int first[kCaRuns + 1];  // places of the runs before it
};
struct CaParts {
    float* acc;  // [2 CTAs][rows][D]: a CTA's part of a unit begun before its range, its part of one that goes on
    float* ml;   // [2 CTAs][rows][2]: maximum (powers of two), sum
    CaList* list;
};
struct CaArgs {
    CUtensorMap keys, values;  // the pools as [rows / 8][d / 64][8][64], in boxes of `box` rows and a slot's values
    CUtensorMap queries;       // [T][Hq][d] in boxes of a tile's tokens, a key head's heads and 64 values
    ChunkAttnArgs a;
    int box;   // rows of a page that are loaded at once: 8 to 128, or 0 (pages not of a multiple of 8): rows one by one
    int span;  // tokens of a tile of rows
    int runs;  // of all sequences, at most (bounds that descend may give more: those are left out)
    int cap;   // keys that may be read
    CaDiv by_page, by_group;
    CaParts parts;
};

// A sequence's tokens and positions.
struct CaSeq {
    int first, tokens;  // of q
    int pos;            // of the first one
    __device__ __forceinline__ CaSeq(const ChunkAttnArgs& a, int s) {
        const bool there = s < a.n;
        first = there ? min(max(a.at[s], 0), a.T) : 0;
        tokens = there ? max(min(a.at[s + 1], a.T) - first, 0) : 0;
        pos = there ? max(a.lens[s], 0) - tokens : 0;
    }
    __device__ __forceinline__ CaSeq() {}
    __device__ __forceinline__ CaSeq of(int lane) const {
        CaSeq o;
        o.first = __shfl_sync(0xffffffffu, first, lane), o.tokens = __shfl_sync(0xffffffffu, tokens, lane), o.pos = __shfl_sync(0xffffffffu, pos, lane);
        return o;
    }
    // runs of `most` tokens
    __device__ __forceinline__ int runs(int most) const { return (tokens + most - 1) / most; }
    // keys that the run's tokens see
    __device__ __forceinline__ int keys(int run, int most, int cap) const { return max(0, min(pos + min((run + 1) * most, tokens), cap)); }
};
__device__ __forceinline__ int ca_tiles(int keys) { return max(1, (keys + kKeys - 1) / kKeys); }

// Lists of a unit's values that are not finite, by k % kOdd: the loads of unit k + 1 and k + 2 may begin while the outputs of unit
// k leave (a short unit's scores end before them). Unit k + 3 is handed out when all warps have taken unit k + 1, so are done with k.
constexpr int kOdd = 3;

constexpr int kUnits = 4;

// What a CTA works on next, handed to all its warps.
struct CaUnit {
    int s, kvh, tok0, toks;  // its tokens, of the sequence's
    int first, pos;          // the sequence's first token in q, its position
    int tile0, tiles, keys;  // tiles 0: no more units
    int whole;
    __device__ __forceinline__ CaUnit() {}
    __device__ __forceinline__ CaUnit(const CaSeq& q, int s, int run, int most, int kvh, int tile0, int tiles, int keys)
        : s(s), kvh(kvh), tok0(run * most), toks(min(most, q.tokens - run * most)), first(q.first), pos(q.pos), tile0(tile0), tiles(tiles), keys(keys), whole(tiles == ca_tiles(keys)) {}
};
// A slot has landed, is free again, has landed but is to be looked through.
template <int kSlots>
struct CaRing {
    unsigned long long full[kSlots], empty[kSlots], raw[kSlots];
};
struct CaBars {
    unsigned long long s_full[2], p_full[2], pv_done[2], o_full[2], o_empty[2], q_full, q_empty, unit_full[2], unit_empty[2], want, stolen, cleared, end;
    uint32_t tmem;
    int bad, polls;
    CaUnit unit[kUnits];                      // handed out two ahead at most; those before them stay for ca_spoil
    __align__(16) uint32_t masks[kMasks][4];  // of a tile's keys, which are there
    uint32_t odd[kOdd][4][4], any_odd[kOdd];  // of a unit's last tiles, keys whose values are not all finite
};

// A wait that gives up after so many polls of 4 us at most, or once another has: the CTA then runs on to its end and makes
// NaN of what it had to do (ca_spoil). Waits are for a tile's work (ChunkAttnArgs::polls, 2^19: two seconds), or for a unit's (2^7 times
// as many): one of 2^30 keys takes ten seconds. No warp waits for another in any other way until the CTA's last barrier.
// After such a wait no warp arrives at a barrier of loads that count their bytes: where one is on its way, an arrival that
// is not due takes the count below 0, which is a fault.
__device__ __forceinline__ bool ca_bad(CaBars& b) { return *reinterpret_cast<volatile int*>(&b.bad) != 0; }
__device__ __forceinline__ bool ca_any_bad(CaBars& b) { return __any_sync(0xffffffffu, ca_bad(b)); }  // (of a warp together)
__device__ __forceinline__ void ca_wait_long(CaBars& b, uint32_t at, uint32_t parity, int polls) {
#pragma unroll 1
    for (int it = 0; it < polls; ++it)
        if (tc::mbar_test_parity(at, parity) || ca_bad(b)) return;
    *reinterpret_cast<volatile int*>(&b.bad) = 1;
}
__device__ __forceinline__ void ca_wait(CaBars& b, unsigned long long* bar, uint32_t parity, bool unit = false) {
    const uint32_t at = tc::smem_addr(bar);
    if (!tc::mbar_test_parity(at, parity)) ca_wait_long(b, at, parity, b.polls << (unit ? 7 : 0));
}
__device__ __forceinline__ void ca_arrive(unsigned long long* bar) { tc::mbar_arrive_cta(tc::smem_addr(bar)); }

// The next unit (the k-th), false: none. Every warp that works on units calls it once a unit.
__device__ __forceinline__ bool ca_next(CaBars& b, uint32_t k, int lane, CaUnit& u) {
    ca_wait(b, &b.unit_full[k & 1], (k >> 1) & 1, true);
    u = b.unit[k % kUnits];
    __syncwarp();
    if (lane == 0) ca_arrive(&b.unit_empty[k & 1]);
    return u.tiles > 0 && !ca_any_bad(b);
}

// The sum over the lanes up to this one.
__device__ __forceinline__ int ca_sum(int x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, x, d);
        if (static_cast<int>(threadIdx.x & 31) >= d) x += o;
    }
    return x;
}

// This CTA's range: f(unit) for each that it has tiles of. CTA i begins at place floor(i total / ctas).
template <int kNQ, class F>
__device__ __forceinline__ void ca_range(const CaArgs& c, const CaList& list, const F& f) {
    const ChunkAttnArgs& a = c.a;
    const int most = kNQ * c.span;
    const int total = list.places * a.Hkv, ctas = min(static_cast<int>(gridDim.x), total), i = blockIdx.x;
    if (i >= ctas) return;
    const int each = total / ctas, rest = total % ctas;
    int at = i * each + i * rest / ctas;
    const int end = (i + 1) * each + (i + 1) * rest / ctas;
    int kvh = at / list.places, off = at % list.places, e = 0, e1 = list.n;
    while (e1 - e > 1) {
        const int mid = (e + e1) / 2;
        (list.first[mid] <= off ? e : e1) = mid;
    }
    off -= list.first[e];
    while (at < end) {
        const int now = min(list.first[e + 1] - list.first[e] - off, end - at), tile0 = max(off - kCaStart, 0), tiles = max(off + now - kCaStart, 0) - tile0;
        const int s = list.unit[e] & 0xFFFFu, run = list.unit[e] >> 16;
        const CaSeq q(a, s);
        if (tiles > 0) f(CaUnit(q, s, run, most, kvh, tile0, tiles, q.keys(run, most, c.cap)));
        at += now, off = 0;
        if (++e == list.n) e = 0, ++kvh;
    }
}

// ---- the warp that hands out units
// kRanges: this CTA's range of all units' tiles. Else units, the longest of a sequence first: that of blockIdx, then those
// of CTAs that have not begun yet, taken over (cancelled) one at a time when the one in work comes to its end, in any order.
template <int kNQ, bool kRanges>
__device__ __forceinline__ void ca_units(const CaArgs& c, CaBars& b, CaList& list, uint4* response) {
    const ChunkAttnArgs& a = c.a;
    const int lane = threadIdx.x & 31, most = kNQ * c.span;
    uint32_t k = 0;
    auto give = [&](const CaUnit& u) {
        ca_wait(b, &b.unit_empty[k & 1], ((k >> 1) - 1) & 1, true);
        if (lane == 0) {
            b.unit[k % kUnits] = u;
            ca_arrive(&b.unit_full[k & 1]);
        }
        ++k;
    };
    auto stop = [&]() {
        ca_wait(b, &b.unit_empty[k & 1], ((k >> 1) - 1) & 1, true);
        if (lane == 0) {
            b.unit[k % kUnits].tiles = 0;
            ca_arrive(&b.unit_full[k & 1]);
        }
    };
    if (kRanges) {
        int n = 0, places = 0;
        for (int s0 = 0; s0 < a.n; s0 += 32) {
            const CaSeq mine(a, s0 + lane);
            const int runs = mine.runs(most);
            const int upto = ca_sum(runs), all = __shfl_sync(0xffffffffu, upto, 31);
            for (int r0 = 0; r0 < all && n < kCaRuns; r0 += 32) {  // a run a lane
                const int r = r0 + lane;
                int src = 0;  // its sequence: the number of those that end before it
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1)
                    if (__shfl_sync(0xffffffffu, upto, src + d - 1) <= r) src += d;
                const CaSeq q = mine.of(src & 31);
                const int run = r - __shfl_sync(0xffffffffu, upto - runs, src & 31);
                const int w = r < all && n + lane < min(c.runs, kCaRuns) ? ca_tiles(q.keys(run, most, c.cap)) + kCaStart : 0, incl = ca_sum(w);
                if (w) list.unit[n + lane] = (s0 + src) | run << 16, list.first[n + lane] = places + incl - w;
                n = min(n + min(all - r0, 32), kCaRuns);
                places += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        n = min(n, min(c.runs, kCaRuns));
        if (lane == 0) list.n = n, list.places = places, list.first[n] = places;
        __syncwarp();
        if (blockIdx.x == 0)  // for the join
            for (int i = lane; i < static_cast<int>(sizeof(CaList) / 4); i += 32) reinterpret_cast<int*>(c.parts.list)[i] = reinterpret_cast<const int*>(&list)[i];
        ca_range<kNQ>(c, list, [&](const CaUnit& u) {
            if (!ca_any_bad(b)) give(u);
        });
        stop();
        return;
    }
    auto of_cta = [&](int id) { return a.backwards ? static_cast<int>(gridDim.x) - 1 - id : id; };
    int unit = of_cta(blockIdx.x), s0 = 0, before = 0;
    CaSeq mine(a, lane);
    uint32_t steals = 0;
    while (true) {
        // the sequence: 32 at a time, on from those of the unit before, or from the first one where that lies behind
        int w, incl;
        if (unit < before) {
            before = 0, s0 = 0;
            mine = CaSeq(a, lane);
        }
        while (true) {
            w = mine.runs(most) * a.Hkv, incl = ca_sum(w);
            const int all = __shfl_sync(0xffffffffu, incl, 31);
            if (unit < before + all || s0 + 32 >= a.n) break;
            before += all, s0 += 32;
            mine = CaSeq(a, s0 + lane);
        }
        const unsigned has = __ballot_sync(0xffffffffu, unit < before + incl);
        if (!has) break;  // past the last unit
        const int src = __ffs(has) - 1, off = unit - before - __shfl_sync(0xffffffffu, incl - w, src);
        const CaSeq q = mine.of(src);
        const int run = q.runs(most) - 1 - off / a.Hkv, keys = q.keys(run, most, c.cap);
        give(CaUnit(q, s0 + src, run, most, off % a.Hkv, 0, ca_tiles(keys), keys));
        ca_wait(b, &b.want, steals & 1, true);
        if (ca_any_bad(b)) break;
        if (lane == 0) {
            tc::fence_proxy_async_smem();
            tc::mbar_arrive_expect_tx(tc::smem_addr(&b.stolen), 16);
            asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(tc::smem_addr(response)),
                         "r"(tc::smem_addr(&b.stolen))
                         : "memory");
        }
        __syncwarp();
        // (whether another wait has given up or not: a unit taken over is this CTA's)
        if (!__all_sync(0xffffffffu, tc::mbar_wait_parity_bounded(tc::smem_addr(&b.stolen), steals & 1, 1 << 19))) {
            *reinterpret_cast<volatile int*>(&b.bad) = 1;
            break;
        }
        ++steals;
        uint32_t got, id;
        asm volatile(
            "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
            : "=r"(got), "=r"(id)
            : "r"(tc::smem_addr(response))
            : "memory");
        if (!got) break;
        unit = of_cta(static_cast<int>(id));
    }
    stop();
}

// ---- the warps that load
// A slot holds 128 keys as groups of 8: [group][64 values][key][128 bytes, swizzled]. 16-byte piece p of key r is at
template <int D>
__device__ __forceinline__ uint32_t ca_at(int r, int p) {
    constexpr uint32_t kChunks = CaCfg<D>::kSlotD / 64;
    return ((r >> 3) * kChunks + (p >> 3)) * 1024 + (r & 7) * 128 + (((p & 7) ^ (r & 7)) << 4);
}

// A unit's queries. (Rows of a box behind the sequence's last token, and those behind a tile's last token, see no key.)
template <int D>
__device__ __forceinline__ void ca_queries(const CaArgs& c, CaBars& b, const CaUnit& u, uint32_t q_smem) {
    if (threadIdx.x % 32 == 0) {
        const int group = c.a.Hq / c.a.Hkv, boxes = (u.toks > c.span ? 2 : 1) * (D / 64);
        tc::mbar_arrive_expect_tx(tc::smem_addr(&b.q_full), boxes * c.span * group * 128);
#pragma unroll 1
        for (int i = 0; i < boxes; ++i)
            asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(q_smem + i * 16384),
                         "l"(&c.queries), "r"(i % (D / 64) * 64), "r"(u.kvh * group), "r"(u.first + u.tok0 + i / (D / 64) * c.span), "r"(tc::smem_addr(&b.q_full))
                         : "memory");
    }
    __syncwarp();
}

// Keys that every row of the unit sees.
__device__ __forceinline__ int ca_common(const CaUnit& u) { return max(0, min(u.pos + u.tok0 + 1, u.keys)); }
// The first tile that not every row sees in full, from the unit's first one.
__device__ __forceinline__ int ca_partly(const CaUnit& u) { return max(ca_common(u) / kKeys - u.tile0, 0); }

// The values of such a tile: a weight of 0 would still carry what is not finite into rows that do not see it (keys of
// later tokens, what lies behind the last one). So it is taken out here, and added at the end where it is seen. A warp's
// rows r0 .. r1 - 1 of a slot (multiples of 8), a 16-byte piece a lane; `odd`: a bit a key of the tile.
template <int DT, int D>
__device__ __forceinline__ void ca_take_odd(uint32_t slot, int r0, int r1, uint32_t* odd, uint32_t* any) {
    constexpr int kPieces = CaCfg<D>::kSlotD / 8;
    const int lane = threadIdx.x & 31, p = lane % kPieces;
    constexpr int kStep = 32 / kPieces, kBatch = 8 / kStep;
    constexpr uint32_t kExp = DT == 1 ? 0x7C00u : 0x7F80u;
#pragma unroll 1
    for (int r = r0 + lane / kPieces; r < r1; r += kBatch * kStep) {
        uint32_t x[kBatch][4], some = 0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                         : "r"(slot + ca_at<D>(r + i * kStep, p))
                         : "memory");
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)  // an exponent of all ones carries out
                some |= ((x[i][e] & 0x7FFF7FFFu) + ((0x8000u - kExp) * 0x10001u)) & 0x80008000u;
        if (some == 0) continue;
#pragma unroll 1
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t at = slot + ca_at<D>(r + i * kStep, p);
            uint32_t y[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]) : "r"(at) : "memory");
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool lo = (y[e] & kExp) == kExp, hi = (y[e] >> 16 & kExp) == kExp;
                hit |= lo | hi;
                if (lo) y[e] &= 0xFFFF0000u;
                if (hi) y[e] &= 0x0000FFFFu;
            }
            if (!hit) continue;
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
            atomicOr(odd + ((r + i * kStep) >> 5), 1u << ((r + i * kStep) & 31));
            *any = 1;
        }
    }
}

// Pages of a multiple of 8 keys: the first warp loads boxes of a page's rows, a lane a box (TMA), the second looks through
// the values of the tiles that are seen in part.
template <int DT, int D, bool kRanges>
__device__ __forceinline__ void ca_load_boxes(const CaArgs& c, CaBars& b, CaRing<CaCfg<D>::kSlots>& bars, uint32_t q_smem, uint32_t ring) {
    using C = CaCfg<D>;
    const ChunkAttnArgs& a = c.a;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - C::kSoftWarps;
    constexpr int kSlots = C::kSlots;
    const int boxes = kKeys / c.box, nowhere = a.n_pages * a.Hkv * a.page;  // (rows behind the pool's last are zeros)
    const int my_box = lane % boxes;
    uint32_t slot = 0, tile = 0, k = 0, phases = 0;
    CaUnit u;
    for (; ca_next(b, k, lane, u); ++k) {
        ca_wait(b, &b.q_empty, (k - 1) & 1, true);
        if (ca_any_bad(b)) return;
        const int partly = ca_partly(u), common = ca_common(u);
        uint32_t* odd = &b.odd[k % kOdd][0][0];
        if (w == 1) {
#pragma unroll 1
            for (int j = partly; j < u.tiles; ++j)
#pragma unroll 1
                for (int p = 0; p < C::kParts; ++p) {
                    // (order of the slots: below)
                    const uint32_t i = slot + p + C::kParts * (C::kNQ == 1 ? min(2 * j + 2, 2 * u.tiles - 1) : 2 * j + 1), at = i % kSlots;
                    ca_wait(b, &bars.raw[at], phases >> at & 1, true);
                    if (ca_any_bad(b)) return;  // (the slot may be another load's)
                    phases ^= 1u << at;
                    // the rows that not all see and that were loaded: the rest of a box behind the last key, no further
                    const int key0 = (u.tile0 + j) * kKeys, r0 = max(common - key0, 0) & ~7, r1 = min((u.keys - key0 + c.box - 1) & -c.box, kKeys);
                    ca_take_odd<DT, D>(ring + at * C::kSlotBytes, r0, r1, odd + 4 * (j - partly), &b.any_odd[k % kOdd]);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ca_arrive(&bars.full[at]);
                }
            slot += 2 * C::kParts * u.tiles;
            continue;
        }
        if (lane < 16) odd[lane] = 0;
        if (lane == 16) b.any_odd[k % kOdd] = 0;
        __syncwarp();
        ca_queries<D>(c, b, u, q_smem);
        const int32_t* table = a.table + static_cast<long long>(u.s) * a.max_pages;
        auto find = [&](int j) -> int {  // this lane's box of tile j: its row in the pools
            const int key = (u.tile0 + j) * kKeys + my_box * c.box;
            if (j >= u.tiles || key >= u.keys) return nowhere;
            const int p = c.by_page(key), pg = table[p];
            return static_cast<unsigned>(pg) < static_cast<unsigned>(a.n_pages) ? (pg * a.Hkv + u.kvh) * a.page + (key - p * a.page) : nowhere;
        };
        // of tile j: its keys, then the values of the tile before it or (two tiles of rows) of its own
        int row = find(0), last = nowhere, next = find(1);
#pragma unroll 1
        for (int j = 0; j < u.tiles + (C::kNQ == 1 ? 1 : 0); ++j) {
            const int later = find(j + 2);
            if (j < u.tiles) {
                const uint32_t on = __ballot_sync(0xffffffffu, row != nowhere);
                if (lane < 4) {
                    uint32_t m = 0;
#pragma unroll
                    for (int g = 0; g < 4; ++g) m |= (on >> (32 * lane + 8 * g) / c.box & 1) * (0xFFu << 8 * g);
                    const int n = u.keys - (u.tile0 + j) * kKeys - 32 * lane;
                    b.masks[(tile + j) % kMasks][lane] = m & (n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1);
                }
                __syncwarp();
            }
#pragma unroll 1
            for (int i = 0; i < 2 * C::kParts; ++i) {
                const bool keys_now = i < C::kParts;
                if (C::kNQ == 1 && (keys_now ? j == u.tiles : j == 0)) continue;
                const int of = C::kNQ == 1 && !keys_now ? j - 1 : j;
                const uint32_t at = slot % kSlots, use = slot / kSlots;
                if (use > 0) ca_wait(b, &bars.empty[at], (use - 1) & 1);
                if (ca_any_bad(b)) return;
                const uint32_t bar = tc::smem_addr(!keys_now && of >= partly ? &bars.raw[at] : &bars.full[at]);
                if (lane == 0) tc::mbar_arrive_expect_tx(bar, C::kSlotBytes);
                __syncwarp();
                if (lane < boxes)
                    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], [%5];" ::"r"(
                                     ring + at * C::kSlotBytes + my_box * c.box * (C::kSlotD * 2)),
                                 "l"(keys_now ? &c.keys : &c.values), "r"(0), "r"((keys_now ? i : i - C::kParts) * (C::kSlotD / 64)),
                                 "r"((of < j ? last : row) >> 3), "r"(bar)
                                 : "memory");
                ++slot;
            }
            if (!kRanges && lane == 0 && j == max(u.tiles - 3, 0)) ca_arrive(&b.want);
            last = row, row = next, next = later;
        }
        tile += u.tiles;
    }
}

// Pages of any size: warp w loads the rows 64 w .. 64 w + 63 of a tile, 16 bytes a lane.
template <int DT, int D, bool kRanges>
__device__ __forceinline__ void ca_load_rows(const CaArgs& c, CaBars& b, CaRing<CaCfg<D>::kSlots>& bars, uint32_t q_smem, uint32_t ring) {
    using C = CaCfg<D>;
    const ChunkAttnArgs& a = c.a;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - C::kSoftWarps;
    constexpr int kPieces = C::kSlotD / 8, kAtOnce = 32 / kPieces, kSlots = C::kSlots;
    const int c8 = lane % kPieces, rr = lane / kPieces;
    uint32_t slot = 0, tile = 0, k = 0;
    int pending = 0;
    uint32_t marks = 0;  // of the slots in flight, oldest lowest, 4 bits each: 1 + which of the unit's last tiles the values are of
    // the slots in flight beyond `keep` have landed
    auto landed = [&](int keep) {
        if (keep) cp_wait<C::kAhead>();
        else cp_wait<0>();
#pragma unroll 1
        for (; pending > keep; --pending, marks >>= 4) {
            const uint32_t at = (slot - pending) % kSlots, mark = marks & 15;
            if (mark) ca_take_odd<DT, D>(ring + at * C::kSlotBytes, 64 * w, 64 * w + 64, b.odd[k % kOdd][mark - 1], &b.any_odd[k % kOdd]);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ca_arrive(&bars.full[at]);
        }
    };
    auto room = [&](unsigned long long* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, tc::mbar_test_parity(tc::smem_addr(bar), parity))) return;
        landed(0);  // the products may wait for these
        ca_wait(b, bar, parity);
    };
    CaUnit u;
    for (; ca_next(b, k, lane, u); ++k) {
        ca_wait(b, &b.q_empty, (k - 1) & 1, true);  // (nothing is in flight)
        if (ca_any_bad(b)) return;
        if (w == 0 && lane < 16) b.odd[k % kOdd][lane >> 2][lane & 3] = 0;
        if (w == 0 && lane == 16) b.any_odd[k % kOdd] = 0;
        __syncwarp();
        if (w == 0) {
            if (lane == 0) ca_arrive(&b.cleared);
            ca_queries<D>(c, b, u, q_smem);
        } else {  // (the first warp clears for unit k + 1 once the scores of unit k, with this warp's keys, are done)
            ca_wait(b, &b.cleared, k & 1, true);
        }
        const int32_t* table = a.table + static_cast<long long>(u.s) * a.max_pages;
        // lane r's rows 64 w + r and 64 w + 32 + r of tile j: their numbers in the pools (-1: not there)
        auto find = [&](int j, int (&row)[2]) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = (u.tile0 + j) * kKeys + 64 * w + 32 * h + lane;
                row[h] = -1;
                if (j < u.tiles && key < u.keys) {
                    const int p = c.by_page(key), pg = table[p];
                    if (static_cast<unsigned>(pg) < static_cast<unsigned>(a.n_pages)) row[h] = (pg * a.Hkv + u.kvh) * a.page + (key - p * a.page);
                }
            }
        };
        const int partly = ca_partly(u);
        // (in the order of the boxes)
        int row[2], last[2] = {-1, -1};
        find(0, row);
#pragma unroll 1
        for (int j = 0; j < u.tiles + (C::kNQ == 1 ? 1 : 0); ++j) {
            int next[2];
            find(j + 1, next);
            if (j < u.tiles) {
                const uint32_t m0 = __ballot_sync(0xffffffffu, row[0] >= 0), m1 = __ballot_sync(0xffffffffu, row[1] >= 0);
                if (lane == 0) b.masks[(tile + j) % kMasks][2 * w] = m0, b.masks[(tile + j) % kMasks][2 * w + 1] = m1;
            }
#pragma unroll 1
            for (int i = 0; i < 2 * C::kParts; ++i) {
                const bool keys_now = i < C::kParts;
                if (C::kNQ == 1 && (keys_now ? j == u.tiles : j == 0)) continue;
                const int of = C::kNQ == 1 && !keys_now ? j - 1 : j;
                const int r0 = of < j ? last[0] : row[0], r1 = of < j ? last[1] : row[1];
                const uint32_t use = slot / kSlots;
                if (use > 0) room(&bars.empty[slot % kSlots], (use - 1) & 1);
                const char* base = static_cast<const char*>(keys_now ? a.k_pool : a.v_pool) + (keys_now ? i : i - C::kParts) * (C::kSlotD * 2) + c8 * 16;
                const uint32_t to = ring + slot % kSlots * C::kSlotBytes;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int from = h ? r1 : r0;
#pragma unroll
                    for (int r = 0; r < 32; r += kAtOnce) {
                        const int n = __shfl_sync(0xffffffffu, from, r + rr);
                        cp16(to + ca_at<D>(64 * w + 32 * h + r + rr, c8), base + static_cast<long long>(max(n, 0)) * (D * 2), n >= 0);
                    }
                }
                cp_commit();
                if (!keys_now && of >= partly) marks |= (of - partly + 1) << (4 * pending);
                ++slot, ++pending;
                if (pending > C::kAhead) landed(C::kAhead);
            }
            if (!kRanges && w == 0 && lane == 0 && j == max(u.tiles - 3, 0)) ca_arrive(&b.want);
#pragma unroll
            for (int h = 0; h < 2; ++h) last[h] = row[h], row[h] = next[h];
        }
        tile += u.tiles;
        landed(0);
    }
}

// ---- the warp that issues the products. All of it keeps step, so that addresses stay in uniform registers (one thread by
// itself takes longer over an instruction's operands than the tensor cores over its product); one lane's count.
__device__ __forceinline__ void ca_mma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool add, bool lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add ? 1u : 0u), "r"(lead ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void ca_mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool add, bool lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add ? 1u : 0u), "r"(lead ? 1u : 0u)
        : "memory");
}
template <int DT, int D>
__device__ __forceinline__ void ca_products(CaBars& b, CaRing<CaCfg<D>::kSlots>& bars, int span, uint32_t q_smem, uint32_t ring) {
    using C = CaCfg<D>;
    constexpr int kNQ = C::kNQ, kParts = C::kParts, kSlots = C::kSlots;
    constexpr uint32_t is = tc::idesc_f16(128, 128, false, false, DT == 2), io = tc::idesc_f16(128, C::kSlotD, false, true, DT == 2);
    // descriptors: addresses in 16 bytes, added to, under constant upper halves
    constexpr uint32_t kChunks = C::kSlotD / 64;
    const uint64_t q_desc = tc::smem_desc(0, 16, 1024, tc::kSwizzle128B), k_desc = tc::smem_desc(0, 16, kChunks * 1024, tc::kSwizzle128B);
    const uint64_t v_desc = tc::smem_desc(0, 1024, kChunks * 1024, tc::kSwizzle128B);
    const uint32_t q_lo = static_cast<uint32_t>(q_desc), q_hi = static_cast<uint32_t>(q_desc >> 32), k_lo = static_cast<uint32_t>(k_desc);
    const uint32_t k_hi = static_cast<uint32_t>(k_desc >> 32), v_lo = static_cast<uint32_t>(v_desc), v_hi = static_cast<uint32_t>(v_desc >> 32);
    const uint32_t q16 = q_smem >> 4, ring16 = ring >> 4;
    const bool lead = (threadIdx.x & 31) == 0;
    uint32_t k_at = 0, v_at = 0, k = 0;           // slots of the current tile's keys and values (of the ring)
    uint32_t next = 0, round = 0;                 // the next slot, and how often the ring has been gone round
    uint32_t k_round = 0, v_round = 0;
    uint32_t soft0 = 0, soft1 = 0, units1 = 0;    // tiles of keys of either tile of rows, units that have the second one
    auto commit = [&](unsigned long long* bar) {
        if (lead) tc::commit(tc::smem_addr(bar));
        __syncwarp();
    };
    auto wait = [&](unsigned long long* bar, uint32_t parity, bool unit = false) {
        ca_wait(b, bar, parity, unit);
        __syncwarp();
        tc::fence_after_sync();
    };
    auto after = [&](uint32_t at, uint32_t& r) {  // the slot behind `at`
        if (++at == kSlots) at = 0, ++r;
        return at;
    };
    auto scores = [&](int q, uint32_t g, bool release) {
        const uint32_t buf = kNQ == 1 ? g & 1 : q, d = C::kScol + 128 * buf;
        uint32_t at = k_at, r = k_round;
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            wait(&bars.full[at], r & 1);
            const uint32_t kb = k_lo + ring16 + at * (C::kSlotBytes / 16), qb = q_lo + q16 + (q * (128 * D * 2) + p * (C::kSlotD / 64) * 16384) / 16;
#pragma unroll
            for (int x = 0; x < C::kSlotD / 16; ++x) {
                ca_mma(d, qb + ((x >> 2) * 16384 + (x & 3) * 32) / 16, q_hi, kb + ((x >> 2) * 1024 + (x & 3) * 32) / 16, k_hi, is, p + x > 0, lead);
            }
            if (release) commit(&bars.empty[at]);
            at = after(at, r);
        }
        commit(&b.s_full[buf]);
    };
    auto values = [&](int q, uint32_t g, int j, uint32_t units, bool last, bool release) {
        const uint32_t buf = kNQ == 1 ? g & 1 : q;
        if (j == 0) wait(&b.o_empty[q], (units - 1) & 1);
        wait(&b.p_full[buf], kNQ == 1 ? (g >> 1) & 1 : g & 1);
        uint32_t at = v_at, r = v_round;
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            wait(&bars.full[at], r & 1);
            const uint32_t vb = v_lo + ring16 + at * (C::kSlotBytes / 16);
#pragma unroll
            for (int x = 0; x < kKeys / 16; ++x)
                ca_mma_ts(q * D + p * 128, C::kScol + 128 * buf + x * 8, vb + x * (kChunks * 2048 / 16), v_hi, io, j > 0 || x > 0, lead);
            if (release) commit(&bars.empty[at]);
            at = after(at, r);
        }
        // A parity tells two phases apart: pv_done of tile j - 1 is asked for while that of j cannot be there yet (its
        // weights are not), and the last one has a barrier of its own.
        commit(last ? &b.o_full[q] : &b.pv_done[q]);
    };
    auto take = [&](uint32_t& at, uint32_t& r) {
        at = next, r = round;
#pragma unroll
        for (int p = 0; p < kParts; ++p) next = after(next, round);
    };
    while (true) {
        wait(&b.unit_full[k & 1], (k >> 1) & 1, true);
        const CaUnit& u = b.unit[k % kUnits];
        const int tiles = __shfl_sync(0xffffffffu, u.tiles, 0), nq = kNQ == 2 && __shfl_sync(0xffffffffu, u.toks, 0) > span ? 2 : 1;
        if (lead) ca_arrive(&b.unit_empty[k & 1]);
        if (tiles <= 0 || ca_any_bad(b)) break;
        wait(&b.q_full, k & 1);
        // one tile of rows: scores of tile j, then values of the one before; two: the values of either, then its scores
        // of the next tile
#pragma unroll 1
        for (int j = kNQ == 1 ? 0 : -1; j < tiles + (kNQ == 1 ? 1 : 0); ++j) {
            if (kNQ == 1) {
                if (j < tiles) {
                    take(k_at, k_round);
                    scores(0, soft0 + j, true);
                    if (j + 1 == tiles) commit(&b.q_empty);
                }
                if (j > 0) {
                    take(v_at, v_round);
                    values(0, soft0 + j - 1, j - 1, k, j == tiles, true);
                }
            } else {
                if (j >= 0) take(v_at, v_round);
                if (j + 1 < tiles) take(k_at, k_round);
#pragma unroll 1
                for (int q = 0; q < nq; ++q) {
                    const uint32_t g = (q ? soft1 : soft0) + j;
                    if (j >= 0) values(q, g, j, q ? units1 : k, j + 1 == tiles, q + 1 == nq);
                    if (j + 1 < tiles) scores(q, g + 1, q + 1 == nq);
                }
                if (j + 2 == tiles) commit(&b.q_empty);
            }
        }
        soft0 += tiles;
        if (nq == 2) soft1 += tiles, ++units1;
        ++k;
    }
    if (ca_any_bad(b)) {
        // a wait gave up: the products in flight still end before tensor memory is given back
        commit(&b.end);
        tc::mbar_wait_parity_bounded(tc::smem_addr(&b.end), 0, 1 << 19);
    }
}

// What was taken out of the values of a unit's last tiles, added to 32 values of a row that sees it.
template <int DT, int D>
__device__ __noinline__ void ca_add_odd(const CaArgs& c, const CaBars& b, const CaUnit& u, uint32_t k, int pos, int col, float* v) {
    const int first = u.tile0 + ca_partly(u);
    for (int i = 0; i < 16; ++i)
        for (uint32_t m = b.odd[k % kOdd][i >> 2][i & 3]; m; m &= m - 1) {
            const int key = (first + (i >> 2)) * kKeys + 32 * (i & 3) + __ffs(m) - 1;
            if (key > pos || key >= u.keys) return;
            const int p = c.by_page(key), pg = c.a.table[static_cast<long long>(u.s) * c.a.max_pages + p];
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(c.a.n_pages)) continue;  // (listed only after a wait that gave up)
            const long long row = (static_cast<long long>(pg) * c.a.Hkv + u.kvh) * c.a.page + (key - p * c.a.page);
            for (int e = 0; e < 32; ++e) {
                const float x = load_act(c.a.v_pool, row * D + col + e, DT);
                if (!(fabsf(x) < INFINITY)) v[e] += x;
            }
        }
}

// 32 bytes of a row: a whole sector each, as neighbouring lanes write other rows (32-byte aligned: rows are, and so is `p`
// where the buffer is; others by halves)
__device__ __forceinline__ void ca_store32(void* p, const uint32_t (&w)[8]) {
    if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                     "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// ---- the weights, one row a thread
template <int DT, int D>
__device__ __forceinline__ void ca_soft(const CaArgs& c, CaBars& b, uint32_t tmem) {
    using C = CaCfg<D>;
    constexpr int kNQ = C::kNQ;
    const ChunkAttnArgs& a = c.a;
    const int r = threadIdx.x, lane = r & 31, q = r >> 7, group = a.Hq / a.Hkv;  // row of the unit, tile of rows
    const uint32_t lanes = static_cast<uint32_t>(r & 96) << 16, o_col = tmem + lanes + q * D;
    const bool flip = a.scale < 0.f;
    // (a scale of 0 is next to 0: masked scores stay -infinity so)
    const float sc = a.scale == 0.f ? 1e-30f : fabsf(a.scale) * kLog2e;
    uint32_t tile = 0, soft = 0, units = 0;  // tiles of keys; those, and units, that have this tile of rows
    const int mine = c.by_group(r & 127), g_head = (r & 127) - mine * group, tok = q * c.span + mine;  // token of the unit, head of the group
    CaUnit u;
    for (uint32_t k = 0; ca_next(b, k, lane, u); ++k, tile += u.tiles) {
        if (q * c.span >= u.toks) continue;
        const bool on = mine < c.span && tok < u.toks;
        const int pos = on ? u.pos + u.tok0 + tok : -1;
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int j = 0; j < u.tiles; ++j) {
            const uint32_t g = soft + j;
            const int buf = kNQ == 1 ? g & 1 : q;
            const uint32_t s_col = tmem + lanes + C::kScol + 128 * buf;
            ca_wait(b, &b.s_full[buf], kNQ == 1 ? (g >> 1) & 1 : g & 1);
            tc::fence_after_sync();
            // keys of the tile that the row sees
            const int lim = pos + 1 - (u.tile0 + j) * kKeys;
            const uint4 there = *reinterpret_cast<const uint4*>(b.masks[(tile + j) % kMasks]);
            if (!__all_sync(0xffffffffu, lim >= kKeys && (there.x & there.y & there.z & there.w) == 0xFFFFFFFFu)) {
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {
                    const int n = lim - 32 * x;
                    const uint32_t see = (x == 0 ? there.x : x == 1 ? there.y : x == 2 ? there.z : there.w) & (n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1);
                    float v[32];
                    tc::tmem_ld32(s_col + 32 * x, v);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = see >> e & 1 ? v[e] : flip ? INFINITY : -INFINITY;
                    tc::tmem_st32(s_col + 32 * x, v);
                }
                tc::tmem_st_wait();
            }
            // all of the row at once: a wait for tensor memory takes hundreds of cycles beside the products
            float v[4][32];
#pragma unroll
            for (int x = 0; x < 4; ++x) tc::tmem_ld32(s_col + 32 * x, v[x]);
            tc::tmem_ld_wait();
            if (flip) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[x][e] = -v[x][e];
            }
            float tops[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                tops[x] = fmaxf(v[x][0], v[x][1]);
#pragma unroll
                for (int e = 2; e < 32; e += 2) tops[x] = fmaxf(tops[x], fmaxf(v[x][e], v[x][e + 1]));
            }
            float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * sc;
            const bool rise = top > m + kTau<DT>;
            if (__any_sync(0xffffffffu, rise)) {
                const float corr = rise ? ex2(m - top) : 1.f;
                if (rise) m = top, l *= corr;
                if (j > 0) {
                    ca_wait(b, &b.pv_done[q], (g - 1 - units) & 1);
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int x = 0; x < D; x += 16) {
                        float o[16];
                        tc::tmem_ld16(o_col + x, o);
                        tc::tmem_ld_wait();
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = __float_as_uint(o[e] * corr);
                        tc::tmem_st16(o_col + x, p);
                    }
                }
            }
            const float back = kUp<DT> - (m == -INFINITY ? 0.f : m);
            const float2 sc2 = make_float2(sc, sc), back2 = make_float2(back, back);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 y = __ffma2_rn(make_float2(v[x][2 * e], v[x][2 * e + 1]), sc2, back2);
                    const float2 w = make_float2(ex2(y.x), ex2(y.y));
                    sum[e & 1] = __fadd2_rn(sum[e & 1], w);
                    p[e] = ca_pack<DT>(w.x, w.y);
                }
                tc::tmem_st16(s_col + 16 * x, p);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ca_arrive(&b.p_full[buf]);
        }
        ca_wait(b, &b.o_full[q], units & 1);
        tc::fence_after_sync();
        const bool odd = *reinterpret_cast<volatile uint32_t*>(&b.any_odd[k % kOdd]) != 0;
        const long long head = static_cast<long long>(u.first + u.tok0 + tok) * a.Hq + u.kvh * group + g_head;
        const long long slot = 2ll * blockIdx.x + (u.tile0 == 0 ? 1 : 0);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
            float v[32];
            tc::tmem_ld32(o_col + x, v);
            tc::tmem_ld_wait();
            if (odd) {
                float w[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = v[e];
                ca_add_odd<DT, D>(c, b, u, k, pos, x, w);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = w[e];
            }
            if (on) {
                if (u.whole) {
                    uint16_t* out = static_cast<uint16_t*>(a.out) + head * D + x;
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = ca_pack<DT>(v[e + 2 * i] * inv, v[e + 2 * i + 1] * inv);
                        ca_store32(out + e, w);
                    }
                } else {
                    float* acc = c.parts.acc + (slot * C::kRows + r) * D + x;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[e + i]);
                        ca_store32(acc + e, w);
                    }
                }
            }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) ca_arrive(&b.o_empty[q]);
        if (on) {
            if (!u.whole) *reinterpret_cast<float2*>(c.parts.ml + (slot * C::kRows + r) * 2) = make_float2(m, l);
            else if (a.lse) a.lse[head] = l == 0.f ? -INFINITY : (m - kUp<DT> + log2f(l)) * kLn2;
        }
        soft += u.tiles, ++units;
    }
}

// After a wait that gave up (one warp): NaN in all that may not be finished or not begun: whole units, of those handed out
// the last ones (a finished one may be among them); ranges, all of this CTA's.
template <int D, bool kRanges>
__device__ __noinline__ void ca_spoil(const CaArgs& c, const CaBars& b, const CaList& list) {
    const ChunkAttnArgs& a = c.a;
    const int lane = threadIdx.x & 31, group = a.Hq / a.Hkv;
    auto spoil = [&](const CaUnit& u) {
        if (!u.whole) {
            for (int r = lane; r < CaCfg<D>::kRows; r += 32)
                *reinterpret_cast<float2*>(c.parts.ml + ((2ll * blockIdx.x + (u.tile0 == 0 ? 1 : 0)) * CaCfg<D>::kRows + r) * 2) = make_float2(0.f, NAN);
            return;
        }
        for (int i = 0; i < u.toks * group; ++i) {
            const int tok = c.by_group(i);
            const long long head = static_cast<long long>(u.first + u.tok0 + tok) * a.Hq + u.kvh * group + (i - tok * group);
            for (int x = lane; x < D / 8; x += 32) reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + head * D)[x] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
            if (lane == 0 && a.lse) a.lse[head] = NAN;
        }
    };
    if (kRanges) {
        ca_range<CaCfg<D>::kNQ>(c, list, spoil);
    } else {
        for (int i = 0; i < kUnits; ++i)
            if (b.unit[i].tiles > 0) spoil(b.unit[i]);
    }
}

template <int DT, int D, bool kRanges>
__global__ void __launch_bounds__(CaCfg<D>::kThreads, 1) chunk_attention_kernel(const __grid_constant__ CaArgs c) {
    using C = CaCfg<D>;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) CaBars b;
    __shared__ CaRing<C::kSlots> bars;
    __shared__ CaList list;
    __shared__ uint4 response;
    const int t = threadIdx.x, warp = t >> 5;
    if (t == 0) {
        auto init = [](unsigned long long* bar, uint32_t count) { tc::mbar_init_cta(tc::smem_addr(bar), count); };
#pragma unroll 1
        for (int i = 0; i < C::kSlots; ++i) init(&bars.full[i], c.box ? 1 : C::kLoadWarps), init(&bars.empty[i], 1), init(&bars.raw[i], 1);
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            init(&b.s_full[i], 1), init(&b.p_full[i], 4), init(&b.pv_done[i], 1), init(&b.o_full[i], 1), init(&b.o_empty[i], 4);
            init(&b.unit_full[i], 1), init(&b.unit_empty[i], C::kSoftWarps + C::kLoadWarps + 1);
        }
        init(&b.q_full, 1), init(&b.q_empty, 1), init(&b.want, 1), init(&b.stolen, 1), init(&b.cleared, 1), init(&b.end, 1);
        b.bad = 0, b.polls = c.a.polls;
#pragma unroll 1
        for (int i = 0; i < kUnits; ++i) b.unit[i].tiles = 0;
        tc::fence_proxy_async_smem();
    }
    if (warp == C::kMmaWarp) {
        tc::tmem_alloc(&b.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_wait();
    pdl_trigger();
    constexpr uint32_t tmem = 0;  // (all of tensor memory is this CTA's)
    const uint32_t q_smem = (tc::smem_addr(raw) + 1023) & ~1023u, ring = q_smem + C::kQBytes;
    // Two tiles of rows: 384 threads begin with 168 registers each, 256 x 200 + 128 x 104 in all.
    if (warp < C::kSoftWarps) {
        if (C::kNQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        ca_soft<DT, D>(c, b, tmem);
    } else {
        if (C::kNQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp < C::kMmaWarp && c.box) ca_load_boxes<DT, D, kRanges>(c, b, bars, q_smem, ring);
        else if (warp < C::kMmaWarp) ca_load_rows<DT, D, kRanges>(c, b, bars, q_smem, ring);
        else if (warp == C::kUnitWarp) ca_units<C::kNQ, kRanges>(c, b, list, &response);
        else ca_products<DT, D>(b, bars, c.span, q_smem, ring);
        __syncwarp();
    }
    // (where a wait gave up: loads in flight land long before this is over)
    if (ca_bad(b))
        for (int i = 0; i < 2000; ++i) __nanosleep(1000);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == C::kMmaWarp) tc::tmem_dealloc(tmem, 512);
    if (warp == C::kUnitWarp && ca_bad(b)) ca_spoil<D, kRanges>(c, b, list);
}

// Joins the parts of the units that lie in several of the `grid` CTAs' ranges. CTA (rows, unit, key head); where the units
// are more than the borders between ranges (by_border), CTA (rows, border), for the unit whose first border that is. Of few
// parts, a warp takes 128 values (64) of a row, eight parts' at once; of many, a CTA does, an eighth of the parts a warp.
constexpr int kCaJoinWarps = 8, kCaAtOnce = 8, kCaFew = 16;
template <int DT, int D>
__global__ void __launch_bounds__(kCaJoinWarps * 32, 4) chunk_attention_join_kernel(const __grid_constant__ CaArgs c, int grid, int by_border) {
    constexpr int kRows = CaCfg<D>::kRows, kVec = D == 64 ? 2 : 4, kSplit = D / (32 * kVec), kWide = 32 * kVec;
    using Vec = std::conditional_t<kVec == 2, float2, float4>;
    __shared__ __align__(16) float sums[kCaJoinWarps][kWide];
    __shared__ float2 mls[kCaJoinWarps][kSms];  // of a row's parts: maximum, then factor; sum
    const ChunkAttnArgs& a = c.a;
    const int group = a.Hq / a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const CaList& list = *c.parts.list;
    const int places = list.places, total = places * a.Hkv, ctas = min(grid, total);
    if (total == 0) return;
    const int each = total / ctas, rest = total % ctas;
    // CTA i begins at place i each + floor(i rest / ctas): place x is CTA x / each's, or one of the few before it
    auto begin = [&](int i) { return i * each + i * rest / ctas; };
    auto owner = [&](int x) {
        int i = min(x / each, ctas - 1);
        while (begin(i) > x) --i;
        return i;
    };
    int e = blockIdx.y, kvh = blockIdx.z;
    if (by_border) {
        if (e + 1 >= ctas) return;
        const int at = begin(e + 1), off = at % places;
        kvh = at / places, e = 0;
        for (int e1 = list.n; e1 - e > 1;) {
            const int mid = (e + e1) / 2;
            (list.first[mid] <= off ? e : e1) = mid;
        }
    } else if (e >= list.n) {
        return;
    }
    const int first = places * kvh + list.first[e] + kCaStart, last = places * kvh + list.first[e + 1] - 1;
    const int c0 = owner(first), n = owner(last) - c0 + 1;
    if (n == 1 || (by_border && c0 != static_cast<int>(blockIdx.y))) return;  // finished, or another border's
    const CaSeq seq(a, list.unit[e] & 0xFFFFu);
    const int tok0 = (list.unit[e] >> 16) * CaCfg<D>::kNQ * c.span, rows = min(CaCfg<D>::kNQ * c.span, seq.tokens - tok0) * group;
    // (many parts: by CTAs only where there are CTAs for all rows: 24 sequences of 8 tokens, up to 21 parts, 15 CTAs a unit: 39 us
    // by warps, 52 by CTAs; one of 16 over 65520 keys, 76 parts, 256 CTAs a unit: 51 and 47)
    const bool few = n <= kCaFew || static_cast<int>(gridDim.x) * 2 < rows * kSplit;
    const int tasks = few ? kCaJoinWarps : 1;  // of a CTA at once
    for (int task = blockIdx.x * tasks + (few ? warp : 0); task < rows * kSplit; task += gridDim.x * tasks) {
        const int pair = task / kSplit, tok = c.by_group(pair), d = (task % kSplit) * kWide + lane * kVec;
        const int r = tok < c.span ? pair : 128 + pair - c.span * group;  // of the unit
        // (a CTA's part of a unit that it begins is its second one)
        auto at = [&](int i) { return (2ll * (c0 + i) + (i == 0 ? 1 : 0)) * kRows + r; };
        float v[kVec] = {}, top = -INFINITY, sum = 0.f;
        // parts i0, i0 + step, ..., kCaAtOnce of them at once; their factors are of the largest maximum
        const int i0 = few ? 0 : warp, step = few ? 1 : kCaJoinWarps;
        __align__(16) float o[kCaAtOnce][kVec];
        auto ahead = [&](int i) {
#pragma unroll
            for (int k = 0; k < kCaAtOnce; ++k)
                if (i + k * step < n) *reinterpret_cast<Vec*>(o[k]) = *reinterpret_cast<const Vec*>(c.parts.acc + at(i + k * step) * D + d);
        };
        ahead(i0);
        for (int i = lane; i < n; i += 32) mls[warp][i] = *reinterpret_cast<const float2*>(c.parts.ml + at(i) * 2);
        for (int i = lane; i < n; i += 32) top = fmaxf(top, mls[warp][i].x);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float base = top == -INFINITY ? 0.f : top;
        for (int i = lane; i < n; i += 32) {
            const float f = ex2(mls[warp][i].x - base);
            mls[warp][i].x = f, sum += mls[warp][i].y * f;
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        __syncwarp();
        for (int i = i0; i < n; i += kCaAtOnce * step) {
#pragma unroll
            for (int k = 0; k < kCaAtOnce; ++k) {
                if (i + k * step >= n) continue;
                const float w = mls[warp][i + k * step].x;
#pragma unroll
                for (int x = 0; x < kVec; ++x) v[x] += o[k][x] * w;
            }
            ahead(i + kCaAtOnce * step);
        }
        __syncwarp();
        if (!few) {
            __syncthreads();
            *reinterpret_cast<Vec*>(&sums[warp][lane * kVec]) = *reinterpret_cast<const Vec*>(v);
            __syncthreads();
            if (warp != 0) continue;
#pragma unroll
            for (int w = 1; w < kCaJoinWarps; ++w)
#pragma unroll
                for (int x = 0; x < kVec; ++x) v[x] += sums[w][lane * kVec + x];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const long long head = static_cast<long long>(seq.first + tok0 + tok) * a.Hq + kvh * group + (pair - tok * group);
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + head * D + d);
        if (kVec == 2) *out = ca_pack<DT>(v[0] * inv, v[1] * inv);
        else *reinterpret_cast<uint2*>(out) = make_uint2(ca_pack<DT>(v[0] * inv, v[1] * inv), ca_pack<DT>(v[kVec - 2] * inv, v[kVec - 1] * inv));
        if (d == 0 && a.lse) a.lse[head] = sum == 0.f ? -INFINITY : (top - kUp<DT> + log2f(sum)) * kLn2;
    }
}

struct CaPlan {
    long long runs;  // at most
    bool ranges;
    int ctas;
    size_t ml, list, total;
};
CaPlan ca_plan(int n, int T, int Hq, int Hkv, int d, int max_len) {
    CaPlan p{};
    const int rows = d == 256 ? 128 : 256, group = Hq / Hkv, most = rows / 128 * (128 / group);
    p.runs = T / most + (n < T ? n : T);
    const long long units = p.runs * Hkv, rounds = (units + kSms - 1) / kSms;
    // Whole units leave CTAs idle in the last round of them, for the time of (rounds 152 - units) / 152 units of the tiles
    // that a unit may have (the host does not know the lengths: an even share of the tokens, behind the longest cache);
    // cut over all CTAs they end together, which costs the parts and a second kernel: 15 us of few units, 30 of many. In
    // tiles of 1.5 us. Whole and cut (16 heads on 2 key heads of 256): 4 tokens over 700 keys 16 and 12 us, 64 over 4064
    // 60 and 29, 256 over 4352 63 and 37, 512 14 and 38, 2048 36 and 65, 2048 behind 8192 242 and 250, behind 14336 392 and
    // 373, behind 30720 788 and 730; 32 heads on 8 of 128, 4096 behind 16384: 1024 and 945.
    // More runs than the list in shared memory has room for stay whole, whatever that costs: sequences of 1 to 4 tokens over
    // up to 16000 keys, 120 of them cut 96 us, 140 whole 232, 200 whole 251 (their bytes: 67, 76, 103).
    const long long tokens = T / n, tiles = (max_len - (tokens < max_len ? tokens : max_len) / 2) / kKeys + 1;
    p.ranges = p.runs <= kCaRuns && (rounds * kSms - units) * tiles > (units < kSms ? 10 : 22) * kSms &&
               units * (max_len / kKeys + 1 + kCaStart) < 1ll << 30;
    p.ctas = kSms;
    if (p.ranges) {
        p.ml = static_cast<size_t>(2) * p.ctas * rows * d * 4;
        p.list = p.ml + static_cast<size_t>(2) * p.ctas * rows * 8;
        p.total = p.list + sizeof(CaList);
    }
    return p;
}
CaDiv ca_div(int d) {
    int l = 0;
    while ((1ll << l) < d) ++l;
    return CaDiv{static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

PFN_cuTensorMapEncodeTiled_v12000 ca_encode() {
    static const PFN_cuTensorMapEncodeTiled_v12000 f = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess) return nullptr;
        return found == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return f;
}
bool ca_map(CUtensorMap* map, const void* p, int dtype, int dims, const cuuint64_t* size, const cuuint64_t* stride, const cuuint32_t* box) {
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const auto encode = ca_encode();
    return encode && encode(map, dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, const_cast<void*>(p), size, stride, box,
                            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool ca_map_pool(CUtensorMap* map, const void* pool, int dtype, int d, int box, const ChunkAttnArgs& a) {
    const cuuint64_t row = static_cast<cuuint64_t>(d) * 2, size[4] = {64, 8, static_cast<cuuint64_t>(d) / 64, static_cast<cuuint64_t>(a.n_pages) * a.Hkv * a.page / 8};
    const cuuint64_t stride[3] = {row, 128, 8 * row};
    const cuuint32_t part[4] = {64, 8, static_cast<cuuint32_t>(d < 128 ? 1 : 2), static_cast<cuuint32_t>(box / 8)};
    return ca_map(map, pool, dtype, 4, size, stride, part);
}
bool ca_map_queries(CUtensorMap* map, int dtype, int d, const ChunkAttnArgs& a) {
    const cuuint64_t size[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.T)};
    const cuuint64_t stride[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(a.Hq) * d * 2};
    const cuuint32_t group = a.Hq / a.Hkv, part[3] = {64, group, 128 / group};
    return ca_map(map, a.q, dtype, 3, size, stride, part);
}

template <int DT, int D>
cudaError_t ca_launch(const ChunkAttnArgs& a, void* ws, cudaStream_t s) {
    using C = CaCfg<D>;
    const CaPlan p = ca_plan(a.n, a.T, a.Hq, a.Hkv, D, a.max_len);
    const long long cap = (long long)a.max_pages * a.page;
    char* w = static_cast<char*>(ws);
    CaArgs c{{}, {}, {}, a, 0, 128 / (a.Hq / a.Hkv), static_cast<int>(p.runs), static_cast<int>(cap < a.max_len ? cap : a.max_len), ca_div(a.page), ca_div(a.Hq / a.Hkv),
             CaParts{reinterpret_cast<float*>(w), reinterpret_cast<float*>(w + p.ml), reinterpret_cast<CaList*>(w + p.list)}};
    if (a.page % 8 == 0) {
        c.box = 8;
        while (c.box < kKeys && a.page % (2 * c.box) == 0) c.box *= 2;
        if (!ca_map_pool(&c.keys, a.k_pool, DT, D, c.box, a) || !ca_map_pool(&c.values, a.v_pool, DT, D, c.box, a)) c.box = 0;
    }
    if (!ca_map_queries(&c.queries, DT, D, a)) return cudaErrorNotSupported;
    const void* f = p.ranges ? reinterpret_cast<const void*>(chunk_attention_kernel<DT, D, true>)
                             : reinterpret_cast<const void*>(chunk_attention_kernel<DT, D, false>);
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    void* args[] = {&c};
    e = launch_kernel(f, dim3(static_cast<unsigned>(p.ranges ? p.ctas : p.runs * a.Hkv)), dim3(C::kThreads), C::kSmem, true, s, args);
    if (e != cudaSuccess || !p.ranges) return e;
    const long long units = p.runs * a.Hkv;
    int grid = p.ctas, by_border = units >= p.ctas;
    // as many CTAs as are on the GPU at once, but no more a unit than it has rows' parts
    const long long most = C::kRows * (D == 256 ? 2 : 1) / (by_border ? kCaJoinWarps : 1), fit = 6 * kSms / (by_border ? p.ctas - 1 : units);
    void* jargs[] = {&c, &grid, &by_border};
    const unsigned x = static_cast<unsigned>(fit < 1 ? 1 : fit < most ? fit : most);
    return launch_kernel(reinterpret_cast<const void*>(chunk_attention_join_kernel<DT, D>),
                         by_border ? dim3(x, p.ctas - 1) : dim3(x, static_cast<unsigned>(p.runs), a.Hkv), dim3(kCaJoinWarps * 32), 0, true, s, jargs);
}

}  // namespace

size_t chunk_attention_ws_bytes(int n, int T, int Hq, int Hkv, int d, int max_len) { return ca_plan(n, T, Hq, Hkv, d, max_len).total; }

cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, int dtype, void* ws, cudaStream_t s) {
    if (dtype == 1) return a.d == 64 ? ca_launch<1, 64>(a, ws, s) : a.d == 128 ? ca_launch<1, 128>(a, ws, s) : ca_launch<1, 256>(a, ws, s);
    return a.d == 64 ? ca_launch<2, 64>(a, ws, s) : a.d == 128 ? ca_launch<2, 128>(a, ws, s) : ca_launch<2, 256>(a, ws, s);
}

}  // namespace escha
