// kda_attn_extend.cu -- chunks of new tokens, of any length each, attend to the paged 8-bit cache, on the 5th-generation
// tensor cores (kda_attention_extend).
//
//   Z = scale ks (Q K^T),  P = 2^(Z log2 e - m),  O = sum P (vs V),  o = O / l        per row, keys in tiles of 128
//
// A unit is one sequence, one key head and up to 256 rows (a group's query heads times 256 / group tokens), in two halves of
// 128; a CTA walks the unit's keys for both.  Codes arrive by bulk copies, a page of a head each, and are converted to f16
// once a tile, exactly (e4m3 and int8 are subsets of f16), by warps that do nothing else.  The products are tcgen05.mma with
// M = 128: Z from Q and K in shared memory, O += P V with P read from tensor memory and V token-major as it lies.  Tensor
// memory: Z0 | Z1 | O0 | O1, P as packed f16 over its Z.  Two threads of the softmax own a row, half of a tile's keys each.
//
// All units' keys, with a gap before each unit for what its start costs, form one line that is cut evenly among the CTAs,
// whatever the lengths are; pieces of a unit are joined by a second kernel in a fixed order.  A unit's key tiles grow with
// its rows' places (causality), so the line is counted in keys, in closed form.
//
// Warps 0-7 and 8-15: softmax of the halves, 16: products, 17: pages and scales, 18-23: conversion (fp32: eight fewer).  They
// meet at mbarriers, each with a limit to its wait: who gives up stops, and with it whoever waits for it, then what is in flight
// is waited for (always with the full limit) and the call's check word tells.
//
// A row of q enters as f16 times a power of two that brings its largest value to [2^14, 2^15): bf16's eight bits are
// exact down to 2^-31 of it.  Weights are held against a reference 2^7 below the row's largest score, which moves only when the
// maximum has grown by more than 2^8, so that they fill f16's range up to 2^15; l sums the unrounded weights in fp32.  V's scales
// enter through P, with O in units that follow the pages' scales.
//
// fp32 io (kSplit): q and the weights as two f16 parts (22 bits), one half of 128 rows; Q's parts take the halves' places and
// so do P's, each with a product of its own.  The products' own sums are cut off, not rounded, so they add one tile's keys
// and ordinary additions the tiles.
//
// Hidden keys: scores are replaced by -inf.  A NaN code in a value would spread over 0 x NaN, so a tile that some row does not see
// whole is cleaned of them (noted by channel and key), and the rows that see them get them at the end.
//
// 2048 tokens behind 30,720 keys, 32 heads of 128 channels over 8: 803 us, 1.33 PFLOP/s (int8 782 us, 1.36), 67 % of the library's
// bf16 products; 256 tokens behind 1,048,320: 3230 us, 1.36 PFLOP/s.  The products alone would take 60 % of a tile's 3400 cycles;
// the rest is the way of a half's tile from scores to weights, which the other half's products do not cover.  What counted
// (the first form took 1813 us): one copy of each role's code, which has to fit a small instruction cache, 1134 -> 943;
// two threads a row, ordinary tiles in one pass over tensor memory, 890; a tile's scales read before its scores arrive; codes by bulk
// copies and not loaded by the converting warps, without a prefetch into L2, 883 -> 797 (with it 909).  Eight warps of
// conversion 919; scores held in registers by one thread a row 950 to 1000.  Few rows: 64 sequences of 4096 keys and one
// token each take 242 us, 2.2 TB/s, bound by conversion and half-empty products (kda_attention_decode takes 100).
// By fits over 8 to 64 tiles a unit: a tile costs an SM 1.6 to 1.9 us, whether 4 rows see it or 256, and a unit's start 3 to 5 us with 4
// rows, 20 with 256.
#include <algorithm>
#include <cfloat>

#include "kda_attn.cuh"
#include "kda_attn_decode.cuh"
#include "kda_attn_tc.cuh"
#include "kda_checks.cuh"

namespace kda {

using namespace attn;

namespace {

constexpr int kKeys = 128;
constexpr int kConvert = 192;
constexpr int kInfo = 8;       // tiles whose pages and scales are known ahead
// The products' warp has a limit of its own, fixed so that it costs nothing: with one from the launch, as the others have, 2048 tokens
// behind 30,720 keys take 2 to 3 % more.
constexpr uint32_t kProductTries = 1u << 16;  // of up to 20 us each
constexpr int kGroups = kKeys / 16;
// What a unit's start and end cost, in keys.  With 128 and 512 long units and many short ones take the same within 1 %, fp32 chunks
// of 333 tokens 43 us with 128 (39 with 256 and 512).
constexpr int kGap = 256;
// Key tiles of a unit that the products add up by themselves.  Their sums are cut off, not rounded, which lowers values of one
// sign: 25,000 steps of 16 keys came out 2.4e-3 low, 2^-23.3 a step.  So what a CTA holds of a unit is a run after the other,
// joined by ordinary additions: of 2^12 steps, 2^-11 of the sum, where half a step of bf16 is 2^-8.  A run's start costs as a unit's
// does, some 25 us: 256 tokens behind 1,048,320 keys take 5 % more with runs of 256 tiles, 2 % with 512.
constexpr int kRun = 512;
constexpr float kUnset = -FLT_MAX;  // the reference of a row that has met no score above -inf
constexpr float kFar = 1048576.f;   // 2^20: references beyond it have their scores rounded first
constexpr uint32_t kHidden = 0xff800000u;
constexpr uint32_t kOdd = 256u;  // some scale of the tile is not a positive finite number, or V's is far below the unit of O
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRestUp = 2048.f;  // what a weight's second part is multiplied by (see kda_attn_decode.cu)

template <int D, bool kSplit> struct Cfg {
    static constexpr int DP = D < 64 ? 64 : D;        // 32 channels are padded with zeros
    static constexpr int NB = DP / 64;                // 64-channel blocks of a row
    static constexpr uint32_t BLK = 128 * 128;        // bytes of a block: 128 rows of 128 bytes
    static constexpr uint32_t TILE = NB * BLK;
    static constexpr int STAGES = D == 128 ? 3 : 6;   // K and V tiles in f16, in turn
    static constexpr int RAWS = D == 128 ? 2 : 4;     // and as codes, on their way or waiting
    static constexpr uint32_t RAW = 128 * D;
    static constexpr uint32_t SMEM = 2 * TILE + STAGES * TILE + RAWS * RAW + 1024;
    static constexpr int HALVES = kSplit ? 1 : 2;
    static constexpr int WARPS = 8 * HALVES;              // of the softmax: a row has two threads, one for each half of a tile's keys
    static constexpr int THREADS = 32 * (WARPS + 8);      // products, pages, six of conversion
    // warpgroups' registers after the split, of what the launch holds
    static constexpr int REGS = kSplit ? 128 : 80, REGS_SOFTMAX = kSplit ? 152 : 88, REGS_OTHER = kSplit ? 104 : 64;
    static_assert(32 * WARPS * REGS_SOFTMAX + 256 * REGS_OTHER <= THREADS * REGS, "register split");
    // tensor memory, columns: where the outputs of the halves (or of P's parts) are, and the sum over tiles (kSplit)
    static constexpr int O = kSplit ? 128 : 256, ACC = 384;
};

// ---------------------------------------------------------------- the line of work

// The new tokens of a sequence that see some key: tokens [start, start + rows) of q, behind `ctx` keys.
struct Seq {
    int64_t start;
    int rows, ctx, skip;  // skip: tokens before them that see none
};

__device__ __forceinline__ Seq seq_of(const AttnExtendArgs& a, int n, bool* bad = nullptr)
{
    int64_t c0, c1;
    if (a.cu != nullptr) {
        c0 = min(max((int64_t)a.cu[n], (int64_t)0), a.T);
        c1 = min(max((int64_t)a.cu[n + 1], c0), a.T);
    } else {
        const int64_t len = a.T / a.N;
        c0 = n * len;
        c1 = c0 + len;
    }
    const int len = a.lengths[n];
    const bool ok = len >= 0 && (int64_t)len <= (int64_t)a.c.max_pages * a.c.page;
    if (!ok && bad != nullptr) *bad = true;
    Seq s;
    const int fresh = (int)(c1 - c0), keys = ok ? len : 0;
    s.skip = max(0, fresh - keys);
    s.start = c0 + s.skip;
    s.rows = fresh - s.skip;
    s.ctx = keys - s.rows;
    return s;
}

// Places of a sequence's units of `tpu` tokens (one key head): a gap and the keys that the last token sees, each.
__device__ __forceinline__ int units_of(const Seq& s, int tpu) { return (s.rows + tpu - 1) / tpu; }
__device__ __forceinline__ int64_t places_before(const Seq& s, int tpu, int64_t k)  // of the units before the k-th
{
    return k * ((int64_t)kGap + s.ctx) + (int64_t)tpu * (k * (k + 1) / 2);
}
__device__ __forceinline__ int64_t places_of(const Seq& s, int tpu)
{
    const int k = units_of(s, tpu);
    return k == 0 ? 0 : places_before(s, tpu, k - 1) + kGap + s.ctx + s.rows;
}

// A run of a unit's key tiles: of those that the CTA holds, which begin with the tile `from`.
struct Segment {
    int n, h, rt, from, i0, count, tiles;
    int first, last, ctx;   // the unit's tokens [first, last) of its sequence's, and the keys before the sequence's first
    int64_t start, place;   // token of q of the sequence's first; where the unit's keys begin in the line
    bool paused;            // the CTA's next run goes on with the unit
    __device__ __forceinline__ bool begun() const { return from == 0; }
    __device__ __forceinline__ bool resumed() const { return i0 > from; }
    __device__ __forceinline__ bool ended() const { return i0 + count == tiles; }
};

// The segments of a CTA, one after the other: the tiles whose first key has its place in [., end).
struct Walk {
    Seq s;
    int n, h, rt, i, from, units;  // from: the unit's first tile here
    int64_t at, end;  // place of the unit's gap
    __device__ __forceinline__ bool next(const AttnExtendArgs& a, int tpu, Segment& g)
    {
        for (;;) {
            if (n >= a.N) return false;
            const int last = min((rt + 1) * tpu, s.rows), keys = s.ctx + last, tiles = (keys - 1) / kKeys + 1;
            const int64_t room = end - (at + kGap + (int64_t)kKeys * i);
            if (i < tiles) {
                if (room <= 0) return false;
                const int left = (int)min((int64_t)(tiles - i), (room + kKeys - 1) / kKeys);
                g.n = n; g.h = h; g.rt = rt; g.from = from; g.i0 = i; g.tiles = tiles;
                g.count = min(left, kRun);
                g.paused = left > kRun;
                g.first = rt * tpu; g.last = last; g.ctx = s.ctx; g.start = s.start; g.place = at + kGap;
                i += g.count;
                return true;
            }
            at += (int64_t)kGap + keys;
            i = from = 0;
            if (++rt < units) continue;
            rt = 0;
            if (++h < a.Hkv) continue;
            h = 0;
            do {
                if (++n >= a.N) return false;
                s = seq_of(a, n);
            } while (s.rows == 0);
            units = units_of(s, tpu);
        }
    }
};

struct Shared {
    uint64_t q_full[2], z_full[2], p_full[2], o_full[2], kv_full[8], kv_empty[8], info_full[kInfo], info_free[kInfo], raw_full[4], raw_free[4], drained;
    uint32_t tmem, dead, flag;
    uint32_t there[kInfo];                                  // bit g: group g of 16 keys is there; and kOdd
    // a tile's scales of K; V's in the unit of O (pv), their logarithm and their reciprocal; the unit, and the last one over it
    alignas(16) float ks[kInfo][kGroups], pv[kInfo][kGroups], lg[kInfo][kGroups], ip[kInfo][kGroups];
    float2 unit[kInfo];
    uint32_t dirty[kInfo];           // by the segment's turn: turn + 1 where something is noted in odd[]
    unsigned long long odd[kInfo][128];  // by the segment's turn: the first key with a NaN in a channel
    Walk begin;     // this CTA's first tile
    Walk walk[24];  // by warp: where it is, and its segment (registers are short)
    Segment seg[24];
    uint32_t more[24];
    float top[2][2][2][128], sum[2][2][2][128];  // in turn: what a row's two threads tell each other, by half and part
    float2 was[2][2][128];                       // in turn: a row's reference and sum where its unit pauses, by half
};

// What is noted in odd[]: the segment's turn in the upper half (later turns are smaller, so that atomicMin prefers them), the
// key in the lower.  A tile's pages are not known before the softmax is done with the tile kInfo before it, and with its segment
// where it was the last: conversion is less than kInfo segments ahead, and as many arrays in turn never mix.
__device__ __forceinline__ unsigned long long odd_note(uint32_t turn, int key)
{
    return ((unsigned long long)(0xfffffffeu - turn) << 32) | (uint32_t)key;
}

// Or over the two warps (64 threads) that share rows; they meet here.
__device__ __forceinline__ bool pair_any(int id, bool x)
{
    uint32_t y;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y)
                 : "r"((uint32_t)x), "r"(id)
                 : "memory");
    return y != 0u;
}

__device__ __forceinline__ float2 f2(float x, float y) { return make_float2(x, y); }

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* v) { KDA_TMEM_LD16(taddr, v); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) { KDA_TMEM_ST16(taddr, v); }

}  // namespace

template <typename TIO, int D, bool kE4m3>
__global__ void __launch_bounds__((Cfg<D, sizeof(TIO) == 4>::THREADS), 1) kda_attn_extend_kernel(const AttnExtendArgs a, const int rows_max, const uint32_t tries)
{
    constexpr bool kSplit = sizeof(TIO) == 4;
    using C = Cfg<D, kSplit>;
    constexpr int S = C::STAGES, kThreads = C::THREADS, kSoft = C::WARPS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    unsigned char* sq = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* ring = sq + 2 * C::TILE;
    unsigned char* raw = ring + S * C::TILE;
    int64_t* prefix = reinterpret_cast<int64_t*>(sq);  // until the work begins
    const int tid = threadIdx.x, lane = tid & 31;
    const int w = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
    const DecodeLayout L = decode_layout(gridDim.x, gridDim.x, rows_max, D);
    const int tpt = 128 / a.group, tpu = C::HALVES * tpt;  // tokens of a half, of a unit
    const int64_t tokrow = (int64_t)a.Hq * D;

    griddep_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.q_full[i], 8);
            tc::mbar_init(&sh.z_full[i], 1);
            tc::mbar_init(&sh.p_full[i], 8);
            tc::mbar_init(&sh.o_full[i], 1);
        }
        for (int i = 0; i < S; ++i) {
            tc::mbar_init(&sh.kv_full[i], kConvert / 32);
            tc::mbar_init(&sh.kv_empty[i], 1);
        }
        for (int i = 0; i < C::RAWS; ++i) {
            tc::mbar_init(&sh.raw_full[i], 1);
            tc::mbar_init(&sh.raw_free[i], kConvert / 32);
        }
        for (int i = 0; i < kInfo; ++i) {
            tc::mbar_init(&sh.info_full[i], 1);
            tc::mbar_init(&sh.info_free[i], kSoft + kConvert / 32);
        }
        tc::mbar_init(&sh.drained, 1);
        sh.dead = 0u;
        sh.flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < kInfo * 128; i += kThreads) (&sh.odd[0][0])[i] = ~0ull;
    if (tid < kInfo) sh.dirty[tid] = 0u;
    if (w == kSoft) tc::tmem_alloc(&sh.tmem, 512);
    // places before every run of `chunk` sequences
    const int chunk = (a.N + kThreads - 1) / kThreads;
    {
        int64_t sum = 0;
        bool bad = false;
        for (int i = 0; i < chunk; ++i) {
            const int n = tid * chunk + i;
            if (n < a.N) sum += places_of(seq_of(a, n, &bad), tpu) * a.Hkv;
        }
        int64_t x = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        prefix[tid + 1] = x;
        if (tid == 0) prefix[0] = 0;
        __syncthreads();
        if (bad) atomicOr(&sh.flag, kCheckBadSeqlens);
        int64_t before = 0;
        for (int i = 0; i < w; ++i) before += prefix[(i + 1) * 32];
        __syncthreads();
        prefix[tid + 1] = x + before;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sh.tmem;
    volatile uint32_t* dead = &sh.dead;

    // tokens that see no key: rows of zeros
    for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
        const Seq s = seq_of(a, n);
        TIO* o = static_cast<TIO*>(a.out) + (s.start - s.skip) * tokrow;
        for (int64_t i = tid; i < s.skip * tokrow; i += kThreads) st_io(o, i, 0.f);
    }
    // This CTA's part of the line.  No more parts than leave each 128 places, so that a unit's middle parts hold a tile each.
    const int64_t total = prefix[kThreads];
    const int64_t W = max((int64_t)1, min((int64_t)gridDim.x, total / kKeys));
    const int64_t b0 = blockIdx.x < W ? blockIdx.x * total / W : total, b1 = blockIdx.x < W ? (blockIdx.x + 1) * total / W : total;
    Walk walk;
    walk.end = b1;
    walk.n = a.N;
    if (b0 < b1) {  // a run of sequences by bisection, then one by one; its head and rows
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= b0) lo = mid;
            else hi = mid - 1;
        }
        int64_t at = prefix[lo], one;
        int n = lo * chunk;
        for (;;) {
            walk.s = seq_of(a, n);
            one = places_of(walk.s, tpu);
            if (at + one * a.Hkv > b0 || n + 1 >= a.N) break;
            at += one * a.Hkv;
            ++n;
        }
        walk.n = n;
        walk.units = units_of(walk.s, tpu);
        walk.h = (int)((b0 - at) / one);
        at += walk.h * one;
        lo = 0;
        hi = walk.units - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at + places_before(walk.s, tpu, mid) <= b0) lo = mid;
            else hi = mid - 1;
        }
        walk.rt = lo;
        walk.at = at + places_before(walk.s, tpu, lo);
        walk.i = walk.from = (int)max((int64_t)0, (b0 - walk.at - kGap + kKeys - 1) / kKeys);
    }
    if (tid == 0) sh.begin = walk;
    __syncthreads();  // the prefix is read
    if constexpr (D < 64) {
        for (int i = tid; i < (int)(S * C::TILE / 16); i += kThreads) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
        tc::fence_async_smem();
        __syncthreads();
    }
    // the warp's next segment
    const Segment& s = sh.seg[w];
    if (lane == 0) sh.walk[w] = walk;
    auto next_segment = [&]() {
        __syncwarp();
        if (lane == 0) sh.more[w] = sh.walk[w].next(a, tpu, sh.seg[w]) ? 1u : 0u;
        __syncwarp();
        return *(volatile uint32_t*)&sh.more[w] != 0u;
    };
    // key tiles of this segment that a half has rows for
    auto tiles_of_half = [&](const Segment& g, int hf) {
        const int first = g.first + hf * tpt;
        if (first >= g.last) return 0;
        const int tiles = (g.ctx + min(first + tpt, g.last) - 1) / kKeys + 1;
        return min(max(tiles - g.i0, 0), g.count);
    };

    if (w >= kSoft) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
        if (w == kSoft + 1) {
            // ---- pages and scales of a tile's groups of 16 keys (lanes 0-7 K's scales, 8-15 V's)
            const int page_shift = 31 - __clz(a.c.page), grp = lane & 7;
            uint32_t t = 0, it = 0;
            bool ok = true;
            while (ok && next_segment()) {
                const int keys = s.ctx + s.last;
                auto page_of = [&](int i) -> int {
                    if (i >= s.i0 + s.count || i * kKeys + grp * 16 >= keys) return -1;
                    const int key = i * kKeys + grp * 16;
                    const int p = __ldg(a.c.table + (int64_t)s.n * a.c.max_pages + (key >> page_shift));
                    return p >= 0 && p < a.c.num_pages ? p : -2;
                };
                const int box = min(kKeys, a.c.page), gpp = box / 16;  // a page's part of a tile, and its groups
                auto scale_of = [&](int p) {
                    return p >= 0 && lane < 16 ? __ldg((lane < 8 ? a.c.k_scale : a.c.v_scale) + (int64_t)p * a.Hkv + s.h) : 0.f;
                };
                // a tile's pages are asked for two tiles ahead, its scales one
                int page = page_of(s.i0), page1 = page_of(s.i0 + 1);
                float vu = 0.f, vtop = 0.f, inv = 0.f;
                float scale = scale_of(page);
                for (int i = s.i0; i < s.i0 + s.count && ok; ++i, ++t) {
                    const int page2 = page_of(i + 2);
                    const float scale1 = scale_of(page1);
                    uint32_t there = __ballot_sync(0xffffffffu, page >= 0) & 0xffu;
                    if (__any_sync(0xffffffffu, page >= 0 && lane < 16 && !(scale > 0.f && scale < INFINITY))) there |= kOdd;
                    if (page == -2) atomicOr(&sh.flag, kCheckBadSeqlens);
                    // The unit of O follows V's scales, from the tile's largest to 64 times it, but never falls under 2^-40 of the
                    // largest met (what is in O would grow past fp32), nor under the smallest with a reciprocal.  Lanes 8-15 have the scales.
                    const uint32_t mag = page >= 0 && lane >= 8 && lane < 16 && fabsf(scale) < INFINITY ? __float_as_uint(fabsf(scale)) : 0u;
                    const float big = __uint_as_float(__reduce_max_sync(0xffffffffu, mag));  // (magnitudes compare as integers)
                    float ratio = 1.f;
                    if (!(big <= vu && big * 64.f >= vu) && big > 0.f) {
                        vtop = fmaxf(vtop, big);
                        const float nu = fmaxf(fmaxf(big, FLT_MIN), vtop * 0x1p-40f);
                        ratio = vu == 0.f ? 0.f : vu / nu;
                        vu = nu;
                        inv = 1.f / vu;
                    }
                    // (a scale's logarithm and reciprocal are those of a power of two, or off by some 2^-22)
                    const float pv = page < 0 ? 1.f : vu == 0.f ? (fabsf(scale) < INFINITY ? 0.f : scale) : scale * inv;
                    const float lg = __log2f(pv), ip = __frcp_rn(pv);
                    // Below 2^-64 weights in the unit of O leave fp32's range, and what their sum gets back from them is not what
                    // went in: such a tile's weights are formed without V's scales, as for scales that have no logarithm.
                    if (__any_sync(0xffffffffu, page >= 0 && lane >= 8 && lane < 16 && fabsf(pv) < 0x1p-64f)) there |= kOdd;
                    const uint32_t slot = t % kInfo;
                    ok = warp_wait(&sh.info_free[slot], ((t / kInfo) & 1u) ^ 1u, tries) && !__any_sync(0xffffffffu, *dead != 0u);
                    if (!ok) break;
                    if (lane < 8) {
                        sh.ks[slot][grp] = scale;
                    } else if (lane < 16) {
                        sh.pv[slot][grp] = pv;
                        sh.lg[slot][grp] = lg;
                        sh.ip[slot][grp] = ip;
                    } else if (lane == 16) {
                        sh.there[slot] = there;
                        sh.unit[slot] = f2(vu, ratio);
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sh.info_full[slot]);
                    // the codes: a page of a head is contiguous, the lane of its first group copies it
                    const int pieces = (__popc(there & 0xffu) + gpp - 1) / gpp;
#pragma unroll 1
                    for (int x = 0; x < 2 && ok; ++x, ++it) {
                        const uint32_t st = it % C::RAWS;
                        ok = warp_wait(&sh.raw_free[st], ((it / C::RAWS) & 1u) ^ 1u, tries);
                        if (!ok) break;
                        if (lane == 0) tc::mbar_arrive_expect_tx(&sh.raw_full[st], (uint32_t)pieces * box * D);
                        __syncwarp();
                        if (lane < 8 && page >= 0 && grp % gpp == 0) {
                            const uint8_t* src = (x ? a.c.v : a.c.k) + (((int64_t)page * a.Hkv + s.h) * a.c.page + ((i * kKeys + grp * 16) & (a.c.page - 1))) * D;
                            tc::bulk_load(raw + st * C::RAW + grp * 16 * D, src, (uint32_t)box * D, &sh.raw_full[st]);
                        }
                    }
                    page = page1;
                    page1 = page2;
                    scale = scale1;
                }
            }
            if (!ok) *dead = 1u;
            // what was issued lands before the CTA ends, also where another role's wait gave up
            if (lane == 0)
                for (uint32_t i = it > (uint32_t)C::RAWS ? it - C::RAWS : 0; i < it; ++i) (void)tc::mbar_wait(&sh.raw_full[i % C::RAWS], (i / C::RAWS) & 1u, kTries);
        } else if (w == kSoft) {
            // ---- products: Z0(0) Z1(0) | O0(0) Z0(1) O1(0) Z1(1) | ...
            const uint32_t f16 = ~((1u << 7) | (1u << 10));
            const uint32_t id_z = tc::idesc_bf16(128, kKeys) & f16, id_o = (tc::idesc_bf16(128, C::DP) & f16) | (1u << 16);
            const uint32_t qa = tc::smem_u32(sq), ra = tc::smem_u32(ring);
            uint32_t it = 0, phase = 0;  // phase: bits 0, 1 of q, 2, 3 of P
            bool ok = true;
            auto full = [&](uint32_t x) { return warp_wait(&sh.kv_full[x % S], (x / S) & 1u, kProductTries); };
            auto flip = [&](uint64_t* bar, uint32_t bit) {
                const bool got = warp_wait(bar, (phase >> bit) & 1u, kProductTries);
                phase ^= 1u << bit;
                return got;
            };
            auto issue_z = [&](int hf, uint32_t x) {
                const uint32_t k = ra + (x % S) * C::TILE;
                // kSplit: both parts of Q into the one Z, the small ones first
#pragma unroll
                for (int p = kSplit ? 1 : 0; p >= 0; --p) {
                    const uint32_t q = qa + (kSplit ? p : hf) * C::TILE;
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) {
                        const uint32_t off = (e >> 2) * C::BLK + (e & 3) * 32;
                        mma_ss(tm + 128 * hf, desc_qk(q + off), desc_qk(k + off), id_z, e > 0 || (kSplit && p == 0));
                    }
                }
                commit(&sh.z_full[hf]);
            };
            auto issue_o = [&](int hf, uint32_t x, bool first) {
                const uint32_t v = ra + (x % S) * C::TILE;
#pragma unroll
                for (int p = 0; p < (kSplit ? 2 : 1); ++p)
#pragma unroll
                    for (int e = 0; e < kKeys / 16; ++e)
                        mma_ts(tm + C::O + C::DP * (kSplit ? p : hf), tm + 128 * hf + (kSplit ? 32 * (e >> 1) + 16 * p + 8 * (e & 1) : 64 * (e >> 2) + 8 * (e & 3)), desc_v(v + e * 2048, D == 128 ? C::BLK : 1024u),
                               id_o, (!kSplit && !first) || e > 0);
            };
            // a slot is given back only after it was seen full, also by a half that has no use for it
            auto release = [&](uint32_t x) { commit(&sh.kv_empty[x % S]); };
            while (ok && next_segment()) {
                const int n0 = tiles_of_half(s, 0), n1 = C::HALVES == 2 ? tiles_of_half(s, 1) : 0, count = s.count;
                // iteration j: the halves' O of tile j, each followed by its Z of tile j + 1 (one copy of either: the roles' code
                // shares a small instruction cache).  V is given back before the last Z, so that the next K has its place early.
#pragma unroll 1
                for (int j = -1; j < count && ok; ++j) {
                    const uint32_t iv = it + 2 * j + 1;
                    const bool more = j + 1 < count;
                    if (j >= 0) ok = full(iv);
#pragma unroll 1
                    for (int hf = 0; hf < C::HALVES && ok; ++hf) {
                        const int nh = hf ? n1 : n0;
                        const bool on = j < nh && nh > 0;
                        if (on) {
                            ok = j < 0 ? flip(&sh.q_full[hf], hf) : flip(&sh.p_full[hf], 2 + hf);
                            if (!ok) break;
                            tc::fence_after_sync();
                            if (j >= 0) issue_o(hf, iv, j == 0);
                        }
                        if (j >= 0 && hf == C::HALVES - 1) release(iv);
                        if (more && hf == 0) ok = full(iv + 1);
                        if (!ok || !on) continue;
                        if (j + 1 < nh) issue_z(hf, iv + 1);  // its commit also covers O's product
                        else commit(&sh.o_full[hf]);
                    }
                    if (!ok) break;
                    if (more) release(iv + 1);
                }
                it += 2 * count;
            }
            if (!ok) *dead = 1u;
            commit(&sh.drained);  // products in flight end before tensor memory is given back
            (void)warp_wait(&sh.drained, 0);
        } else {
            // ---- conversion: 16 codes a thread at a time, into the products' layout
            constexpr int RC = D / 16;  // 16-code pieces of a row
            constexpr int kTurns = (kKeys * RC + kConvert - 1) / kConvert;
            const int me = tid - 32 * (kSoft + 2);
            // 128 channels: sixteen lanes take two rows, eight of them half of each, so that their 16-byte stores, which the
            // layout puts at even places of one row and odd places of the other, fill the banks once
            constexpr int kStep = kConvert / RC;  // rows from a thread's piece to its next: multiples of 8
            const int row0 = RC == 8 ? 2 * (me >> 4) + ((me >> 2) & 1) : me / RC;
            const int ch = RC == 8 ? (me & 3) + 4 * (((me >> 2) ^ (me >> 3)) & 1) : me % RC;
            static_assert(kConvert % RC == 0 && kStep % 8 == 0, "a thread's pieces lie in one column of the layout");
            unsigned char* const to = ring + (ch >> 2) * C::BLK + row0 * 128;
            const int c0 = ((2 * ch) & 7) ^ (row0 & 7), c1 = c0 ^ 1;
            const uint32_t from = row0 * D + ch * 16;
            uint32_t t = 0, it = 0, turn = 0;  // tile, item (K or V of a tile), segment
            bool ok = true;
            auto inside = [&](int e) { return (e + 1) * kStep <= kKeys || row0 + kStep * e < kKeys; };
            for (; ok && next_segment(); ++turn) {
                const int keys = s.ctx + s.last, hidden = s.ctx + s.first + 1, end = s.i0 + s.count;  // hidden: the first key that some row does not see
#pragma unroll 1
                for (int i = s.i0; i < end && ok; ++i, ++t) {
                    const int key0 = i * kKeys;
                    uint32_t there = 0u;
#pragma unroll 1
                    for (int x = 0; x < 2; ++x, ++it) {
                        const uint32_t rs = it % C::RAWS, st = it % S;
                        ok = warp_wait(&sh.raw_full[rs], (it / C::RAWS) & 1u, tries);
                        if (!ok) break;
                        if (x == 0) there = sh.there[t % kInfo] & 0xffu;
                        uint4 u[kTurns];
#pragma unroll
                        for (int e = 0; e < kTurns; ++e)
                            if (inside(e)) u[e] = *reinterpret_cast<const uint4*>(raw + rs * C::RAW + from + e * kStep * D);
                        if (there != 0xffu || key0 > keys - kKeys) {  // keys that are not there
#pragma unroll
                            for (int e = 0; e < kTurns; ++e) {
                                const int row = row0 + kStep * e;
                                if (key0 + row >= keys || ((there >> (row >> 4)) & 1u) == 0u) u[e] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                        if (kE4m3 && x && key0 > hidden - kKeys) {  // NaN that not every row may see leave the tile
#pragma unroll
                            for (int e = 0; e < kTurns; ++e) {
                                uint32_t c[4] = {u[e].x, u[e].y, u[e].z, u[e].w};
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const uint32_t nan = inside(e) ? __vcmpeq4(c[q] & 0x7f7f7f7fu, 0x7f7f7f7fu) : 0u;
                                    if (nan == 0u) continue;
#pragma unroll 1
                                    for (int b = 0; b < 4; ++b)
                                        if ((nan >> (8 * b)) & 1u)
                                            atomicMin(&sh.odd[turn % kInfo][ch * 16 + q * 4 + b], odd_note(turn, key0 + row0 + kStep * e));
                                    sh.dirty[turn % kInfo] = turn + 1u;
                                    c[q] &= ~nan;
                                }
                                u[e] = make_uint4(c[0], c[1], c[2], c[3]);
                            }
                        }
                        ok = warp_wait(&sh.kv_empty[st], ((it / S) & 1u) ^ 1u, tries);
                        if (!ok) break;
                        unsigned char* dst = to + st * C::TILE;
#pragma unroll
                        for (int e = 0; e < kTurns; ++e) {
                            if (!inside(e)) continue;
                            uint32_t h[8];
                            widen<kE4m3>(u[e].x, h[0], h[1]);
                            widen<kE4m3>(u[e].y, h[2], h[3]);
                            widen<kE4m3>(u[e].z, h[4], h[5]);
                            widen<kE4m3>(u[e].w, h[6], h[7]);
                            *reinterpret_cast<uint4*>(dst + e * kStep * 128 + c0 * 16) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4*>(dst + e * kStep * 128 + c1 * 16) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                        tc::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tc::mbar_arrive(&sh.kv_full[st]);
                            tc::mbar_arrive(&sh.raw_free[rs]);
                            if (x == 0) tc::mbar_arrive(&sh.info_free[t % kInfo]);
                        }
                    }
                }
            }
            if (!ok) *dead = 1u;
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
        // ---- softmax: two warpgroups have half hf, a row (of a tensor-memory lane) two threads: `part` 0 has keys 0-63 of a tile and the
        // first half of the channels, 1 the others
        const int hf = w >> 3, part = (w >> 2) & 1, r = tid & 127;
        const int pair = 1 + 4 * hf + (w & 3);           // their warps' barrier
        const uint32_t lanes = (uint32_t)(w & 3) << 21;  // lane offset 32 (w % 4) in the address' upper half
        const uint32_t zt = tm + 128 * hf + 64 * part + lanes, ot = tm + C::O + C::DP * hf + D / 2 * part + lanes;
        const uint32_t at = tm + C::ACC + D / 2 * part + lanes;
        const int rt = r / a.group, rh = r - rt * a.group;
        uint32_t zc = 0, oc = 0, t = 0, turn = 0, told = 0;
        bool gone = false;
        for (; !gone && next_segment(); ++turn) {
            const int nh = tiles_of_half(s, hf);
            const int tok = s.first + hf * tpt + rt;
            const bool on = rt < tpt && tok < s.last;
            float cs = 0.f;
            if (nh > 0) {
                // the row of q, scaled by a power of two, into the products' layout (the half's last products have ended); each thread
                // half of the channels
                const TIO* q = static_cast<const TIO*>(a.q) + (s.start + tok) * a.qs + (int64_t)(s.h * a.group + rh) * D + D / 2 * part;
                constexpr int kWords = D / 2 * (int)sizeof(TIO) / 16, kBatch = kWords < 8 ? kWords : 8;
                float mx = 0.f;
#pragma unroll 1
                for (int c = 0; c < kWords; c += kBatch) {
                    uint4 u[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) u[i] = on ? __ldg(reinterpret_cast<const uint4*>(q) + c + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const uint32_t y[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (kSplit) mx = fmaxf(mx, fabsf(f_of(y[e])));
                            else mx = max3(mx, fabsf(f_of(y[e] << 16)), fabsf(f_of(y[e] & 0xffff0000u)));
                        }
                    }
                }
                told ^= 1u;
                sh.top[told][hf][part][r] = mx;
                (void)pair_any(pair, false);
                mx = fmaxf(mx, sh.top[told][hf][part ^ 1][r]);
                const int e = min(max((int)((__float_as_uint(mx) >> 23) & 0xffu) - 127, -100), 127);
                const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);  // 2^(14 - e)
                cs = __uint_as_float((uint32_t)(127 + e - 14) << 23) * a.scale * kLog2e;
#pragma unroll 2
                for (int i = 0; i < C::DP / 16; ++i) {  // (again, from L1)
                    // 8 channels; those past D are zeros
                    const int c = i < D / 16 ? D / 16 * part + i : D / 8 + (C::DP - D) / 16 * part + i - D / 16;
                    uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
                    if (on && i < D / 16) {
                        float x[8];
                        if constexpr (kSplit) {
                            const float4 y = __ldg(reinterpret_cast<const float4*>(q) + 2 * i), v = __ldg(reinterpret_cast<const float4*>(q) + 2 * i + 1);
                            x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w; x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
                        } else {
                            const uint4 v = __ldg(reinterpret_cast<const uint4*>(q) + i);
                            const uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                x[2 * b] = f_of(y[b] << 16);
                                x[2 * b + 1] = f_of(y[b] & 0xffff0000u);
                            }
                        }
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float x0 = x[2 * b] * up, x1 = x[2 * b + 1] * up;
                            hi[b] = pack_f16(x0, x1);
                            if constexpr (kSplit) {
                                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[b]));
                                lo[b] = pack_f16(x0 == f.x ? 0.f : x0 - f.x, x1 == f.y ? 0.f : x1 - f.y);  // (an infinity has no rest)
                            }
                        }
                    }
                    const uint32_t to = (c >> 3) * C::BLK + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                    *reinterpret_cast<uint4*>(sq + hf * C::TILE + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (kSplit) *reinterpret_cast<uint4*>(sq + C::TILE + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                tc::fence_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.q_full[hf]);
            }
            const int seen = on ? s.ctx + tok + 1 : INT32_MAX;  // keys that the row sees
            const int warp_seen = __reduce_min_sync(0xffffffffu, seen);
            float m = kUnset, vu = 0.f, l = 0.f;  // m: finite, so that a score of -inf weighs nothing
            float peak = -INFINITY;               // the largest weight's exponent among ordinary tiles since m was set (this thread's)
            const int count = s.count, i0 = s.i0;
            bool late = false, left = false;  // a wait gave up, here or with the row's other thread: they leave together
            for (int j = 0; j < count; ++j, ++t) {
                const int slot = t % kInfo;
                if (j < nh) {
                    late = !warp_wait(&sh.z_full[hf], zc++ & 1u, tries);
                    tc::fence_after_sync();
                    if constexpr (kSplit) {
                        // the last tile's outputs, both parts, to the sum of those before it (their products ended with the scores)
                        if (j > 0) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o0[16], o1[16], ac[16];
                                tmem_ld16(ot + 16 * c, o0);
                                tmem_ld16(ot + C::DP + 16 * c, o1);
                                if (j > 1) tmem_ld16(at + 16 * c, ac);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float x = fmaf(f_of(o1[i]), 1.f / kRestUp, f_of(o0[i]));
                                    ac[i] = __float_as_uint(j > 1 ? f_of(ac[i]) + x : x);
                                }
                                tmem_st16(at + 16 * c, ac);
                            }
                            tc::tmem_wait_st();
                        }
                    }
                    const uint32_t there = sh.there[slot];
                    const float2 unit = sh.unit[slot];
                    vu = unit.x;
                    const int key0 = (i0 + j) * kKeys;
                    auto k_of = [&](int c) {  // at least FLT_MIN where all scales are positive numbers: -inf times it stays that
                        const float2 x = *reinterpret_cast<const float2*>(&sh.ks[slot][4 * part + 2 * c]);
                        return (there & kOdd) != 0u ? f2(x.x * cs, x.y * cs) : f2(fmaxf(x.x * cs, FLT_MIN), fmaxf(x.y * cs, FLT_MIN));
                    };
                    auto store = [&](const uint32_t (&p)[16], const uint32_t (&p1)[kSplit ? 16 : 1], int c) {
                        tmem_st16(zt + (kSplit ? 32 : 16) * c, p);
                        if constexpr (kSplit) tmem_st16(zt + 32 * c + 16, p1);
                    };
                    auto pack = [&](float2 y, uint32_t& hi, uint32_t& lo) {
                        hi = pack_f16(y.x, y.y);
                        if constexpr (kSplit) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                            lo = pack_f16((y.x - f.x) * kRestUp, (y.y - f.y) * kRestUp);
                        }
                    };
                    // A weight has its value's scale in the exponent (2^(score + log2 pv - m), it comes off the sums group by group).
                    // In an ordinary tile none passes 2^15, which is found out on the way; P, which goes over Z, waits for that.  (What
                    // decides is the same for both threads of a row.)
                    bool ordinary = j > 0 && there == 0xffu && key0 <= warp_seen - kKeys && unit.y == 1.f && !__any_sync(0xffffffffu, fabsf(m) > kFar);
                    if (ordinary) {
                        uint32_t z[32], p[2][16], p1[2][kSplit ? 16 : 1];
                        float over = -INFINITY, sums = 0.f;
                        tmem_ld32(zt, z);
                        const float2 kgs[2] = {k_of(0), k_of(1)};
                        const float4 lgs = *reinterpret_cast<const float4*>(&sh.lg[slot][4 * part]), ips = *reinterpret_cast<const float4*>(&sh.ip[slot][4 * part]);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float2 kg = kgs[c], lg = c ? f2(lgs.z, lgs.w) : f2(lgs.x, lgs.y), ip = c ? f2(ips.z, ips.w) : f2(ips.x, ips.y);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float k = i < 8 ? kg.x : kg.y, off = (i < 8 ? lg.x : lg.y) - m;
                                const float2 x = __ffma2_rn(f2(f_of(z[2 * i]), f_of(z[2 * i + 1])), f2(k, k), f2(off, off));
                                z[2 * i] = __float_as_uint(x.x);
                                z[2 * i + 1] = __float_as_uint(x.y);
                                over = max3(over, x.x, x.y);
                            }
                            float2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 y = f2(ex2(f_of(z[2 * i])), ex2(f_of(z[2 * i + 1])));
                                sum[i >> 3] = __fadd2_rn(sum[i >> 3], y);
                                pack(y, p[c][i], p1[c][kSplit ? i : 0]);
                            }
                            if (c == 0) tmem_ld32(zt + 32, z);
                            sums = fmaf(sum[0].x + sum[0].y, ip.x, sums);
                            sums = fmaf(sum[1].x + sum[1].y, ip.y, sums);
                            if (c == 0) tc::tmem_wait_ld();
                        }
                        ordinary = !pair_any(pair, over > 15.f || late);
                        if (ordinary) {
                            l += sums;
                            peak = fmaxf(peak, over);
                            store(p[0], p1[0], 0);
                            store(p[1], p1[1], 1);
                        }
                    }
                    if (!ordinary) {
                        // Any tile: hidden scores leave Z, the largest weight, the weights.  References move to 2^7 below the largest
                        // weight here, not only where it has passed 2^15 but wherever it has grown by more than 2^2: what one row
                        // makes necessary then serves its warp's others, whose turn would come one by one.  A row beyond 2^20, where a
                        // score's rounding would show (and all rows where a scale is no positive number), has its scores rounded, as
                        // the reference is, before it comes off, so that none passes the largest however large they are, and the
                        // value's scale is multiplied with.
                        if (key0 > warp_seen - kKeys || (there & 0xffu) != 0xffu) {
#pragma unroll 1
                            for (int c = 0; c < 2; ++c) {
                                uint32_t z[32];
                                const int n = seen - key0 - 64 * part - 32 * c;
                                const uint32_t first = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u, g = there >> (4 * part + 2 * c);
                                const uint32_t see = first & ((g & 1u ? 0xffffu : 0u) | (g & 2u ? 0xffff0000u : 0u));
                                tmem_ld32(zt + 32 * c, z);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if ((see & (1u << i)) == 0u) z[i] = kHidden;
                                tmem_st32(zt + 32 * c, z);
                            }
                            tc::tmem_wait_st();
                        }
                        bool own = (there & kOdd) != 0u, some = own;
                        float now = m;
                        for (int round = some ? 1 : 0;; ++round) {
                            float top = -INFINITY;
#pragma unroll 1
                            for (int c = 0; c < 2; ++c) {
                                uint32_t z[32];
                                tmem_ld32(zt + 32 * c, z);
                                const float2 kg = k_of(c), lg = *reinterpret_cast<const float2*>(&sh.lg[slot][4 * part + 2 * c]);
                                tc::tmem_wait_ld();
                                if (round == 0) {
#pragma unroll
                                    for (int g = 0; g < 2; ++g) {
                                        const uint32_t* x = z + 16 * g;
                                        float m0 = fmaxf(f_of(x[0]), f_of(x[1])), m1 = fmaxf(f_of(x[2]), f_of(x[3]));
#pragma unroll
                                        for (int i = 4; i < 16; i += 4) {
                                            m0 = max3(m0, f_of(x[i]), f_of(x[i + 1]));
                                            m1 = max3(m1, f_of(x[i + 2]), f_of(x[i + 3]));
                                        }
                                        top = fmaxf(top, fmaf(fmaxf(m0, m1), g ? kg.y : kg.x, g ? lg.y : lg.x));
                                    }
                                } else {
#pragma unroll
                                    for (int i = 0; i < 32; ++i) {
                                        const float y = __fmul_rn(f_of(z[i]), i < 16 ? kg.x : kg.y);
                                        if (z[i] != kHidden) top = fmaxf(top, y);
                                    }
                                }
                            }
                            told ^= 1u;
                            sh.top[told][hf][part][r] = round == 0 ? fmaxf(top, m + peak) : top;
                            left = pair_any(pair, late);
                            if (left) break;
                            top = fmaxf(sh.top[told][hf][0][r], sh.top[told][hf][1][r]);
                            if (round == 0 || own) now = (m == kUnset && top > -INFINITY) || top - m > (own ? 15.f : 9.f) ? top - 7.f : m;
                            if (round == 1) break;
                            own = (fabsf(m) > kFar && m != kUnset) || (fabsf(now) > kFar && now != kUnset);
                            some = __any_sync(0xffffffffu, own);
                            if (!some) break;
                        }
                        if (left) break;
                        const float alpha = now == m ? 1.f : ex2(m - now), f = alpha * unit.y;  // O's unit may have changed, too
                        peak -= now - m;
                        m = now;
                        l *= alpha;
                        if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                const uint32_t to = (kSplit ? at : ot) + 16 * c;
                                uint32_t o[16];
                                tmem_ld16(to, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(f_of(o[i]) * f);
                                tmem_st16(to, o);
                            }
                        }
                        const float ref = m == kUnset ? 0.f : m;
                        float sums = 0.f;
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t z[32], p[16], p1[kSplit ? 16 : 1];
                            tmem_ld32(zt + 32 * c, z);
                            const float2 kg = k_of(c), lg = *reinterpret_cast<const float2*>(&sh.lg[slot][4 * part + 2 * c]);
                            const float2 ip = *reinterpret_cast<const float2*>(&sh.ip[slot][4 * part + 2 * c]);
                            tc::tmem_wait_ld();
                            if (some) {
                                // this row's own scores less the reference; the others' scores as they are
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float y = __fsub_rn(__fmul_rn(f_of(z[i]), i < 16 ? kg.x : kg.y), ref);
                                    if (own) z[i] = z[i] == kHidden ? kHidden : __float_as_uint(y);
                                }
                            }
                            float2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
                            const float2 pv = *reinterpret_cast<const float2*>(&sh.pv[slot][4 * part + 2 * c]);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float k = own ? 1.f : i < 8 ? kg.x : kg.y, off = own ? 0.f : (i < 8 ? lg.x : lg.y) - ref;
                                float2 y = __ffma2_rn(f2(f_of(z[2 * i]), f_of(z[2 * i + 1])), f2(k, k), f2(off, off));
                                y = f2(ex2(y.x), ex2(y.y));
                                sum[i >> 3] = __fadd2_rn(sum[i >> 3], y);
                                if (some && own) {  // (a hidden key's scale may be no number)
                                    const float v = i < 8 ? pv.x : pv.y;
                                    y = f2(y.x == 0.f ? 0.f : y.x * v, y.y == 0.f ? 0.f : y.y * v);
                                }
                                pack(y, p[i], p1[kSplit ? i : 0]);
                            }
                            sums = fmaf(sum[0].x + sum[0].y, own ? 1.f : ip.x, sums);
                            sums = fmaf(sum[1].x + sum[1].y, own ? 1.f : ip.y, sums);
                            store(p, p1, c);
                        }
                        l += sums;
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sh.p_full[hf]);
                } else {
                    // (not before the tile is known: the barrier still counts the slot's last one)
                    late = !warp_wait(&sh.info_full[slot], (t / kInfo) & 1u, tries) || __any_sync(0xffffffffu, *dead != 0u);
                    if (late) {  // once for all of the segment's tiles; the row's threads meet below
                        *dead = 1u;
                        break;
                    }
                }
                // the last tile's when the segment is over: conversion then is less than kInfo segments ahead (see odd_note)
                __syncwarp();
                if (lane == 0 && j + 1 < count) tc::mbar_arrive(&sh.info_free[slot]);
            }
            if (!left) {
                if (nh > 0 && !late) late = !warp_wait(&sh.o_full[hf], oc++ & 1u, tries);
                sh.sum[turn & 1][hf][part][r] = l;
                left = pair_any(pair, late || *dead != 0u);
            }
            gone = left;
            if (gone) break;
            tc::fence_after_sync();
            l += sh.sum[turn & 1][hf][part ^ 1][r];
            const bool whole = s.begun() && s.ended();
            const int64_t place = (2 * (int64_t)blockIdx.x + (s.begun() ? 1 : 0)) * rows_max + hf * 128 + r;
            // a piece is a mean, too: sums of large values would pass fp32's range (and vu / l could fall under it)
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // What the unit's earlier runs left here, and the weights of this one and of those in what both give.
            const bool resumed = s.resumed();
            float now = 1.f, then = 0.f;
            if (resumed) {
                const float2 was = sh.was[(turn & 1) ^ 1][hf][r];
                const float both = fmaxf(m, was.x), l1 = l * ex2(m - both), l0 = was.y * ex2(was.x - both);
                m = both;
                l = l1 + l0;
                now = l == 0.f ? 0.f : l1 / l;
                then = l == 0.f ? 0.f : l0 / l;
            }
            if (s.paused && part == 0) sh.was[turn & 1][hf][r] = f2(m, l);
            TIO* out = static_cast<TIO*>(a.out) + (s.start + tok) * tokrow + (int64_t)(s.h * a.group + rh) * D + D / 2 * part;
            float* po = reinterpret_cast<float*>(a.ws + L.o) + place * D + D / 2 * part;
            if (on && !whole && part == 0) reinterpret_cast<float2*>(a.ws + L.ml)[place] = make_float2(m, l);
            const bool dirty = kE4m3 && *(volatile uint32_t*)&sh.dirty[turn % kInfo] == turn + 1u;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[16];
                if (nh > 0) {
                    tmem_ld16(ot + 16 * c, o);
                    if constexpr (kSplit) {
                        uint32_t o1[16], ac[16];
                        tmem_ld16(ot + C::DP + 16 * c, o1);
                        if (nh > 1) tmem_ld16(at + 16 * c, ac);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float x = fmaf(f_of(o1[i]), 1.f / kRestUp, f_of(o[i]));
                            o[i] = __float_as_uint(nh > 1 ? f_of(ac[i]) + x : x);
                        }
                    } else {
                        tc::tmem_wait_ld();
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0u;
                }
                if (!on) continue;
                float y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = f_of(o[i]) * inv * vu;
                if (dirty) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const unsigned long long od = sh.odd[turn % kInfo][D / 2 * part + 16 * c + i];
                        if ((uint32_t)(od >> 32) == 0xfffffffeu - turn && (int)(uint32_t)od < seen) y[i] = NAN;
                    }
                }
                if (resumed) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(po + 16 * c + 4 * i);
                        y[4 * i] = fmaf(y[4 * i], now, x.x * then);
                        y[4 * i + 1] = fmaf(y[4 * i + 1], now, x.y * then);
                        y[4 * i + 2] = fmaf(y[4 * i + 2], now, x.z * then);
                        y[4 * i + 3] = fmaf(y[4 * i + 3], now, x.w * then);
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(po + 16 * c + 4 * i) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                } else if constexpr (kSplit) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(out + 16 * c + 4 * i) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                } else {
                    uint32_t b[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[i] = tc::pack_bf16(y[2 * i], y[2 * i + 1]);
                    *reinterpret_cast<uint4*>(out + 16 * c) = make_uint4(b[0], b[1], b[2], b[3]);
                    *reinterpret_cast<uint4*>(out + 16 * c + 8) = make_uint4(b[4], b[5], b[6], b[7]);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.info_free[(t - 1) % kInfo]);
        }
        if (gone) *dead = 1u;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (w == kSoft) tc::tmem_dealloc(tm, 512);
    if (tid == 0) {
        // what this CTA leaves to be joined: the unit that it began and did not end
        Record rec{-1, 0, 0, 0, 0};
        const bool failed = sh.dead != 0u;
        Walk walk = sh.begin;
        Segment s;
        while (walk.next(a, tpu, s)) {
            if (failed || s.paused || !s.begun() || s.ended()) continue;
            const int64_t e = s.place + (int64_t)kKeys * (s.tiles - 1);  // the last tile's place
            rec = Record{s.n, s.h, s.rt, (int32_t)blockIdx.x, (int32_t)(((e + 1) * W - 1) / total)};
        }
        reinterpret_cast<Record*>(a.ws + L.records)[blockIdx.x] = rec;
        reinterpret_cast<uint32_t*>(a.ws + L.flags)[blockIdx.x] = sh.flag | (failed ? kCheckTimeout : 0u);
    }
}

// Joins a unit's pieces: o = sum_i w_i o_i / sum_i w_i, w_i = 2^(m_i - m) l_i, over the CTAs that hold one, in an order that the
// pieces' number fixes.  m: the largest m_i + floor(log2 l_i) and 10 more, so that no weight passes 2^-9, nor 512 pieces' sum the
// largest value (beyond scores of 2^24, which have no room for that logarithm, values have to stay below 2^70).  `wpr` warps take a row's pieces in turn; a block takes kJoinWarps / wpr rows of a unit at a
// time: block (x, y) those of the unit that CTA x began or, where few CTAs have begun one (kFew), of the units in turn.
constexpr int kJoinWarps = 8;
constexpr int kMaxWorkers = 512;

template <typename TIO, int D, bool kFew>
__global__ void __launch_bounds__(kJoinWarps * 32)
    kda_attn_extend_join_kernel(const AttnExtendArgs a, const int rows_max, const int workers, const int tpu, const int half_tokens, const int wpr)
{
    constexpr int V = D / 32;
    __shared__ float part[kJoinWarps][D + 1];
    __shared__ int units[kFew ? kMaxWorkers : 1];  // the CTAs that began a unit which they did not end, in order
    __shared__ int counts[kJoinWarps];
    __shared__ uint32_t word;
    const DecodeLayout L = decode_layout(workers, workers, rows_max, D);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    griddep_wait();
    const Record* records = reinterpret_cast<const Record*>(a.ws + L.records);
    int count = 0;
    for (int base = 0; kFew && base < workers; base += kJoinWarps * 32) {
        const int i = base + threadIdx.x;
        const uint32_t yes = __ballot_sync(0xffffffffu, i < workers && records[i].n >= 0);
        if (lane == 0) counts[w] = __popc(yes);
        __syncthreads();
        int before = count;
        for (int x = 0; x < kJoinWarps; ++x) {
            before += x < w ? counts[x] : 0;
            count += counts[x];
        }
        if ((yes >> lane) & 1u) units[before + __popc(yes & ((1u << lane) - 1u))] = i;
        __syncthreads();
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        // the call's check word: every CTA's flags, so that nothing has to be cleared before the call
        if (threadIdx.x == 0) word = 0u;
        __syncthreads();
        uint32_t f = 0u;
        const uint32_t* flags = reinterpret_cast<const uint32_t*>(a.ws + L.flags);
        for (int i = threadIdx.x; i < workers; i += blockDim.x) f |= flags[i];
        if (f) atomicOr(&word, f);
        __syncthreads();
        if (threadIdx.x == 0) *reinterpret_cast<uint32_t*>(a.ws) = word;
    }
    const int rows = kJoinWarps / wpr, turns = (rows_max + rows - 1) / rows;  // rows at a time, times for a unit
    for (int item = blockIdx.x; !kFew || item < count * turns; item += gridDim.x) {
        const Record rec = records[kFew ? units[item / turns] : blockIdx.x];
        if (!kFew && rec.n < 0) return;
        const Seq s = seq_of(a, rec.n);
        const int r = (kFew ? item % turns : blockIdx.y) * rows + w / wpr;  // row of the unit: 128 a half
        const int in_half = r & 127, tok = rec.rt * tpu + (r >> 7) * half_tokens + in_half / a.group;
        const bool on = r < rows_max && in_half < half_tokens * a.group && tok < min((rec.rt + 1) * tpu, s.rows);
        const float2* ml = reinterpret_cast<const float2*>(a.ws + L.ml);
        const float* po = reinterpret_cast<const float*>(a.ws + L.o);
        const int pieces = rec.last - rec.first + 1;
        auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * rec.first + 1 : 2 * (rec.first + i)); };
        float l = 0.f, o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.f;
        if (on) {
            float m = -FLT_MAX;
            for (int i = lane; i < pieces; i += 32) {
                const float2 x = ml[slot(i) * rows_max + r];
                m = fmaxf(m, x.x + (float)((int)(__float_as_uint(x.y) >> 23) - 117));
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll 4
            for (int i = w % wpr; i < pieces; i += wpr) {
                const float2 x = ml[slot(i) * rows_max + r];
                const float* p = po + (slot(i) * rows_max + r) * D + lane * V;
                const float f = x.y * ex2(x.x - m);
                l += f;
                if constexpr (V == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(p);
                    o[0] += y.x * f; o[1] += y.y * f; o[2] += y.z * f; o[3] += y.w * f;
                } else if constexpr (V == 2) {
                    const float2 y = *reinterpret_cast<const float2*>(p);
                    o[0] += y.x * f; o[1] += y.y * f;
                } else {
                    o[0] += *p * f;
                }
            }
        }
        if (wpr > 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) part[w][lane * V + v] = o[v];
            if (lane == 0) part[w][D] = l;
            __syncthreads();
            for (int i = 1; i < wpr && w % wpr == 0; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] += part[w + i][lane * V + v];
                l += part[w + i][D];
            }
            if (kFew) __syncthreads();  // (read before the next rows' replace it)
        }
        if (!on || w % wpr != 0) {
            if constexpr (kFew) continue;
            else return;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        TIO* od = static_cast<TIO*>(a.out) + ((s.start + tok) * a.Hq + rec.h * a.group + in_half % a.group) * D + lane * V;
#pragma unroll
        for (int v = 0; v < V; ++v) st_io(od, v, o[v] * inv);
        if (!kFew) return;
    }
}

namespace {

int extend_ctas() { return std::min(sm_count_of_current_device(), kMaxWorkers); }

// Rows of a piece: a unit's, or fewer where the call has no more in one half.
int piece_rows(int64_t tokens, int group, kda_dtype_t dt)
{
    const int64_t half = 128 / group;
    return tokens > half && dt == KDA_BF16 ? 256 : tokens >= half ? 128 : (int)(tokens * group);
}

template <typename TIO, int D, bool kE4m3>
cudaError_t launch_extend(const AttnExtendArgs& a, cudaStream_t s)
{
    constexpr bool kSplit = sizeof(TIO) == 4;
    using C = Cfg<D, kSplit>;
    static_assert(C::SMEM + sizeof(Shared) <= 232448, "the tiles fit an SM");
    auto kern = kda_attn_extend_kernel<TIO, D, kE4m3>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    const int ctas = extend_ctas();
    const int rows = piece_rows(a.T, a.group, kSplit ? KDA_F32 : KDA_BF16);
    kern<<<ctas, C::THREADS, C::SMEM, s>>>(a, rows, checks::handoff_tries(kTries));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // About ctas / units pieces a unit: four or more a warp.  Where a quarter of the CTAs at most can have begun a unit (one for
    // every token tile and sequence), no more blocks than their rows need or an SM holds: 4 units in 32 pieces take 24.6 us with
    // these and 38.5 with blocks for every CTA's every row; 150 units 806 with these and 800 with all.
    const int half_tokens = 128 / a.group, tpu = C::HALVES * half_tokens;
    const int64_t units = (a.T + tpu - 1) / tpu * a.Hkv, pieces = ctas / units;
    const int wpr = pieces >= 32 ? 8 : pieces >= 16 ? 4 : pieces >= 8 ? 2 : 1;
    const int64_t most = (a.T / tpu + std::min<int64_t>(a.T, a.N)) * a.Hkv, turns = (rows * wpr + kJoinWarps - 1) / kJoinWarps;
    if (most <= ctas / 4) {
        const int64_t blocks = std::min<int64_t>(most * turns, 8LL * ctas);
        return launch_dependent(kda_attn_extend_join_kernel<TIO, D, true>, dim3((unsigned)blocks), dim3(kJoinWarps * 32), 0, s, a, rows, ctas, tpu, half_tokens, wpr);
    }
    return launch_dependent(kda_attn_extend_join_kernel<TIO, D, false>, dim3((unsigned)ctas, (unsigned)turns), dim3(kJoinWarps * 32), 0, s, a, rows, ctas, tpu, half_tokens, wpr);
}

template <typename TIO, int D>
cudaError_t launch_code(const AttnExtendArgs& a, cudaStream_t s)
{
    return a.c.dtype == KDA_CACHE_E4M3 ? launch_extend<TIO, D, true>(a, s) : launch_extend<TIO, D, false>(a, s);
}

template <typename TIO>
cudaError_t launch_d(const AttnExtendArgs& a, cudaStream_t s)
{
    return a.d == 32 ? launch_code<TIO, 32>(a, s) : a.d == 64 ? launch_code<TIO, 64>(a, s) : launch_code<TIO, 128>(a, s);
}

}  // namespace

size_t attn_extend_workspace_bytes(int64_t tokens, int group, int d, kda_dtype_t dt)
{
    const int ctas = extend_ctas();
    return decode_layout(ctas, ctas, piece_rows(tokens, group, dt), d).total;
}

cudaError_t launch_attn_extend(const AttnExtendArgs& a, kda_dtype_t dt, cudaStream_t s)
{
    if (a.T == 0) return cudaMemsetAsync(a.ws, 0, 4, s);  // the check word
    return dt == KDA_BF16 ? launch_d<__nv_bfloat16>(a, s) : launch_d<float>(a, s);
}

}  // namespace kda
