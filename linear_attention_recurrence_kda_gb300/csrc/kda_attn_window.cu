// kda_attn_window.cu -- many rows a key head over the paged 8-bit cache, on the 5th-generation tensor
// cores (kda_attention_decode: a drafted window, a large group of query heads; bf16, 128 channels).
//
//   Z^T = scale ks (K Q^T),  P = 2^(Z - m),  O^T = sum V^T P^T,  o = O / l        as in kda_attn_decode.cu
//
// With 28 rows a key head the warp-level kernel spends about 1300 instructions on a tile of 32 keys, most
// of them conversions and products.  Here a CTA takes up to 32 rows and keys in blocks of 128: the
// codes are converted once, by warps that do nothing else, into f16 tiles (exactly: e4m3 and int8 are
// subsets of f16), from which tcgen05.mma forms Z^T (keys are the product's 128 rows, queries its 32
// columns) and O^T (channels the rows).  A thread of the softmax then owns a key and its 32 scores: no lane
// is idle, a key's scales are the thread's own, and no score crosses lanes but at a change of the
// reference.  Few columns make the products cheap (about 128 cycles each a block).
//
// What bounds it: of an SM's cycles at work, loads and stores keep the path to shared memory busy 49 %, the
// products' reads 22 %; a unit's start and end cost as much as 5 blocks (64 sequences of 300 to 6000 keys, 28
// rows of 8 heads: 134 us with the join, 3.1 TB/s, where HBM would allow 62).
//
// Blocks alternate between two streams, each with its own reference, sums and O, so that one's softmax
// runs while the other waits; at the end of a unit the first stream joins them.  Tensor memory: Z0 | Z1 |
// O0 | O1, 32 columns each; P goes through shared memory.  All units' blocks, with a gap before each unit for
// what its start costs, form one line that is cut evenly among the CTAs; pieces of a unit are joined by the join kernel.
//
// Warps 0-3 and 4-7: softmax of the streams, 8: products, 9: copies and scales, 10-15: conversion.  A row of
// q enters scaled by a power of two that its own largest value sets, so that what one row holds, a NaN
// or an infinity too, changes no other; V's scales enter through P, with O in units of the block's
// largest scale.  Weights enter as f16, up to 2^15, with the reference 2^7 below the largest (see kda_attn_decode.cu).
#include <cfloat>
#include <type_traits>

#include "kda_attn.cuh"
#include "kda_attn_decode.cuh"
#include "kda_attn_tc.cuh"

namespace kda {

using namespace attn;

namespace {

constexpr int kBlk = 128;  // keys per block
constexpr int kRows = 32;  // rows of a unit: the products' columns
constexpr int kThreads = 512;
constexpr int kConvert = 192;
constexpr int kRaw = 4;    // raw tiles (K and V in turn) on their way or waiting
constexpr int kGroups = kBlk / 16;
// What a unit's start and end cost (q, the first references, the streams' join), in blocks.  Cut by blocks alone,
// the CTAs that hold short sequences end last: SMs were at work 70 % of the time, now 92 %.  28 rows of 8 heads,
// us for a cost of 0, 3, 5, 10: 64 sequences of 300 to 6000 keys 174, 140, 134, 141; 200 of 100 to 900
// 196, 138, 132, 138; 256 of 256 to 600 173, 160, 158, 161; 64 of 3150 134, 132, 133, 134.
constexpr int kUnitCost = 5;
// warpgroups' registers after the split: 256 x 168 + 256 x 88 = 512 x 128, what the launch holds
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = 0x1p-11f;  // products, which stay below 2^31, may pass 2^20 as scores by a factor above this

constexpr int D = 128;
constexpr uint32_t kColBlk = 128 * 128;         // bytes of 64 channels of 128 keys in f16
constexpr uint32_t kTileBytes = 2 * kColBlk;    // a K or V block in f16
constexpr uint32_t kQBlk = kRows * 128;         // 64 channels of the rows of q
constexpr uint32_t kQBytes = 2 * kQBlk;
constexpr uint32_t kPBytes = kBlk * kRows * 2;  // P^T: a key's 32 weights are 64 bytes
constexpr uint32_t kRawBytes = kBlk * D;        // a block of codes
constexpr uint32_t kSmem = kQBytes + 2 * kPBytes + 4 * kTileBytes + kRaw * kRawBytes + 1024;  // K and V twice

struct Shared {
    uint64_t raw_full[kRaw], raw_free[kRaw], k_ready[2], k_free[2], v_ready[2], v_free[2];
    uint64_t q_ready, f_read, z_full[2], p_full[2], o_full[2], joined, join_free, drained;
    uint32_t tmem, dead, flag;
    uint32_t has[8];             // by block: bit g, group g of 16 keys is there
    float ks[8][kGroups], vs[8][kGroups];
    alignas(16) float f[kRows];  // a row's scores are in units of 2^s (see row_unit)
    uint32_t mixed;              // is some row's unit another than 1?
    float top[2][4][kRows];      // by stream and warp: the largest score of a row
    float sum[2][4][kRows];      // a row's sum
    alignas(16) float ref[2][kRows], by[2][kRows];  // a row's reference, and what its last change multiplies by
    float unit[2];
    int64_t at[kRows];           // where a row's output goes
    float weight[2][kRows];      // the streams' weights in a row's result
    unsigned long long odd[4][128];  // by the segment's turn: the first key with a NaN in a channel (see odd_note)
    Cursor begin;                // this CTA's first block
    int left;                    // and its part of the line from there on
};

// A run of a unit's blocks.
struct Segment {
    int n, h, rt, i0, count, len;
    bool begun, ended;  // does it hold the unit's first block, its last?
};

// the segments of a worker, one after the other
struct Walk {
    Cursor c;
    int left;  // of the line, from block c on
    int gap;   // of the line before a unit's first block
    __device__ __forceinline__ bool next(const AttnDecodeArgs& a, int row_tiles, Segment& s)
    {
        if (left <= 0) return false;
        s.n = c.n; s.h = c.h; s.rt = c.rt; s.i0 = c.i; s.len = c.len;
        s.count = min(left, c.tiles - c.i);
        s.begun = c.i == 0;
        s.ended = c.i + s.count == c.tiles;
        left -= s.count + gap;
        if (left > 0) {
            c.i = c.tiles - 1;
            next_tile<kBlk>(a, row_tiles, c);
        }
        return true;
    }
};

// P^T as the second operand, rows contiguous: 64-byte rows of one key, groups of 8 keys 512 bytes apart,
// 64-byte swizzle.  V as the first operand, channels contiguous.
constexpr uint32_t kDescHi64 = (512u >> 4) | (1u << 14) | (4u << 29);
__device__ __forceinline__ void mma_vp(uint32_t d, uint32_t a_lo, uint32_t b_addr, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(((b_addr & 0x3FFFFu) >> 4) | (1u << 16)), "r"(idesc), "r"(kDescHi), "r"(kDescHi64), "r"((uint32_t)accumulate)
        : "memory");
}

// The power of two s (of s = 16 c) for rows of q whose largest magnitude lies in [2^(16 c - 8), 2^(16 c + 8)); such a row
// enters as f16 times 2^(7 - s).  Rows of one c, as a model's are, share their scores' unit, and scores need no
// factor of their row (one for every row, 64 sequences of 300 to 6000 keys, 28 rows of 8 heads: 142 us against
// 134).  The largest value lands in [2^-1, 2^15): bf16's eight bits are exact down to 2^-16 of it at worst, and
// what is cut off below that is at most 2^-24 of it, like an fp32 sum's last place.
__device__ __forceinline__ int row_unit(uint32_t top)  // the bits of the largest magnitude; zeros: 0
{
    const int e = min(max((int)(top >> 7) - 127, -100), 127);
    return top == 0u ? 0 : min((e + 8) >> 4 << 4, 127);  // the last: 2^127, and its values land below 2^8
}

// Or over the 128 threads of a stream (its four warps meet here).
__device__ __forceinline__ bool any4(int stream, bool x)
{
    uint32_t y;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y)
                 : "r"((uint32_t)x), "r"(1 + stream)
                 : "memory");
    return y != 0u;
}

// Lane r's result of reducing x[r] over the warp: each step halves the values a lane still holds.
template <typename F>
__device__ __forceinline__ float reduce_rows(float (&x)[32], F f)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float give = up ? x[i] : x[i + off];
            const float keep = up ? x[i + off] : x[i];
            x[i] = f(keep, __shfl_xor_sync(0xffffffffu, give, off));
        }
    }
    return x[0];
}

// A noted NaN: the segment's turn in the upper half (later turns are smaller, so that atomicMin prefers
// them), the key's distance from the last key that every row sees in the lower.  Conversion is at
// most two segments ahead of the softmax, so four arrays in turn never mix.
__device__ __forceinline__ unsigned long long odd_note(uint32_t turn, int key, int last)
{
    return ((unsigned long long)(0xfffffffeu - turn) << 32) | (uint32_t)max(key - last, 0);
}

}  // namespace

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1)
    kda_attn_window_kernel(const AttnDecodeArgs a, const int rows_max, const bool by_unit)
{
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    unsigned char* sk = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sv = sk + 2 * kTileBytes;   // two (and K's two)
    unsigned char* sq = sv + 2 * kTileBytes;
    unsigned char* sp = sq + kQBytes;          // two
    unsigned char* raw = sp + 2 * kPBytes;     // kRaw
    int64_t* prefix = reinterpret_cast<int64_t*>(raw);  // until the copies begin
    const int tid = threadIdx.x, lane = tid & 31;
    const int w = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
    const DecodeLayout L = decode_layout(gridDim.x, gridDim.x, rows_max, D);
    const int rows_all = a.L * a.group;
    const int row_tiles = (rows_all + kRows - 1) / kRows;
    const int64_t per_block = (int64_t)a.Hkv * row_tiles;
    const int64_t tokrow = (int64_t)a.Hq * D;

    griddep_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kRaw; ++i) {
            tc::mbar_init(&sh.raw_full[i], 1);
            tc::mbar_init(&sh.raw_free[i], kConvert / 32);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.k_ready[i], kConvert / 32);
            tc::mbar_init(&sh.k_free[i], 1);
            tc::mbar_init(&sh.v_ready[i], kConvert / 32);
            tc::mbar_init(&sh.v_free[i], 1);
            tc::mbar_init(&sh.z_full[i], 1);
            tc::mbar_init(&sh.p_full[i], 4);
            tc::mbar_init(&sh.o_full[i], 1);
        }
        tc::mbar_init(&sh.q_ready, 4);
        tc::mbar_init(&sh.f_read, 4);
        tc::mbar_init(&sh.joined, 4);
        tc::mbar_init(&sh.join_free, 4);
        tc::mbar_init(&sh.drained, 1);
        sh.dead = 0u;
        sh.flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 4 * 128; i += kThreads) (&sh.odd[0][0])[i] = ~0ull;
    if (w == 8) tc::tmem_alloc(&sh.tmem, 128);
    // The line that is cut evenly: each unit takes a place for every block, after a gap for what its start and
    // end cost (where there are fewer units than CTAs, every piece has a start: no gap).
    const int gap = by_unit ? 0 : kUnitCost;
    auto places_of = [&](int tiles) { return tiles > 0 ? tiles + gap : 0; };
    // places before every run of `chunk` sequences
    const int chunk = (a.N + kThreads - 1) / kThreads;
    {
        int64_t sum = 0;
        bool bad = false;
        for (int i = 0; i < chunk; ++i) {
            const int n = tid * chunk + i;
            if (n < a.N) sum += places_of(tiles_of<kBlk>(length_of(a, n, &bad)));
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
    Record* records = reinterpret_cast<Record*>(a.ws + L.records);
    auto unit_of = [&](const Segment& s) { return (int64_t)s.n * per_block + (int64_t)s.h * row_tiles + s.rt; };

    // a sequence with nothing in the cache: rows of zeros
    for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
        if (length_of(a, n) == 0) {
            for (int i = tid; by_unit && i < per_block; i += kThreads) records[n * per_block + i].n = -1;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (int64_t)n * a.L * tokrow;
            for (int64_t i = tid; i < a.L * tokrow; i += kThreads) o[i] = __float2bfloat16_rn(0.f);
        }
    }
    const int64_t total = prefix[kThreads] * per_block;
    const int64_t W = min((int64_t)gridDim.x, total);
    const int64_t b0 = blockIdx.x < W ? blockIdx.x * total / W : 0, b1 = blockIdx.x < W ? (blockIdx.x + 1) * total / W : 0;
    Walk walk;
    auto start = [&]() {  // at this CTA's first block: a run of sequences by bisection, then one by one
        walk.left = (int)(b1 - b0);
        walk.gap = gap;
        walk.c = Cursor{0, 0, 0, 0, 1, 0};
        if (walk.left <= 0) return;
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] * per_block <= b0) lo = mid;
            else hi = mid - 1;
        }
        int64_t at = prefix[lo] * per_block;
        Cursor& c = walk.c;
        c.n = lo * chunk;
        for (;;) {
            c.len = length_of(a, c.n);
            c.tiles = tiles_of<kBlk>(c.len);
            const int64_t here = places_of(c.tiles) * per_block;
            if (at + here > b0 || c.n + 1 >= a.N) break;
            at += here;
            ++c.n;
        }
        const int64_t rest = b0 - at, unit = rest / places_of(c.tiles);
        const int place = (int)(rest - unit * places_of(c.tiles));
        c.i = max(0, place - gap);
        walk.left -= max(0, gap - place);
        c.h = (int)(unit / row_tiles);
        c.rt = (int)(unit - (int64_t)c.h * row_tiles);
    };
    start();
    if (tid == 0) {
        sh.begin = walk.c;
        sh.left = walk.left;
    }
    tc::fence_async_smem();  // the copies take over where the prefix was
    __syncthreads();
    Segment s;

    if (w >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (w == 9) {
            // ---- copies of codes, and the scales of a block's groups of 16 keys (lanes 0-7 K's, 8-15 V's)
            const int box = min(kBlk, a.c.page), gpp = box / 16;
            const int page_shift = 31 - __clz(a.c.page);
            const int grp = lane & 7;
            uint32_t it = 0, blk = 0;
            auto page_of = [&](const Segment& g, int i) -> int {
                const int key = i * kBlk + grp * 16;
                if (key >= g.len) return -1;
                const int p = __ldg(a.c.table + (int64_t)g.n * a.c.max_pages + (key >> page_shift));
                return p >= 0 && p < a.c.num_pages ? p : -2;
            };
            auto scale_of = [&](const Segment& g, int p) {
                return p >= 0 && lane < 16 ? __ldg((lane < 8 ? a.c.k_scale : a.c.v_scale) + (int64_t)p * a.Hkv + g.h) : 0.f;
            };
            bool ok = true;
            while (ok && walk.next(a, row_tiles, s)) {
                // a block's pages are asked for two blocks ahead, its scales one
                int page = page_of(s, s.i0), page1 = s.count > 1 ? page_of(s, s.i0 + 1) : -1;
                float scale = scale_of(s, page);
                for (int i = s.i0; i < s.i0 + s.count && ok; ++i, ++blk) {
                    const int page2 = i + 2 < s.i0 + s.count ? page_of(s, i + 2) : -1;
                    const float scale1 = scale_of(s, page1);
                    const uint32_t there = __ballot_sync(0xffffffffu, page >= 0) & 0xffu;
                    if (page == -2) atomicOr(&sh.flag, kCheckBadSeqlens);
                    for (int x = 0; x < 2 && ok; ++x, ++it) {
                        const uint32_t st = it % kRaw;
                        ok = warp_wait(&sh.raw_free[st], ((it / kRaw) & 1u) ^ 1u);
                        if (!ok) break;
                        if (x == 0) {
                            if (lane < 8) sh.ks[blk & 7][grp] = scale;
                            else if (lane < 16) sh.vs[blk & 7][grp] = scale;
                            if (lane == 0) sh.has[blk & 7] = there;
                            __syncwarp();
                        }
                        const int pieces = __popc(there) / gpp + (__popc(there) % gpp != 0 ? 1 : 0);
                        if (lane == 0) tc::mbar_arrive_expect_tx(&sh.raw_full[st], (uint32_t)pieces * box * D);
                        // a page of a head is contiguous: the lane of its first group copies it
                        __syncwarp();
                        if (lane < 8 && page >= 0 && grp % gpp == 0) {
                            const uint8_t* src = (x ? a.c.v : a.c.k) +
                                                 (((int64_t)page * a.Hkv + s.h) * a.c.page + ((i * kBlk + grp * 16) & (a.c.page - 1))) * D;
                            tc::bulk_load(raw + st * kRawBytes + grp * 16 * D, src, (uint32_t)box * D, &sh.raw_full[st]);
                        }
                    }
                    page = page1;
                    page1 = page2;
                    scale = scale1;
                }
            }
            if (!ok) *dead = 1u;
            if (lane == 0 && *dead)
                for (uint32_t i = it > kRaw ? it - kRaw : 0; i < it; ++i) (void)tc::mbar_wait(&sh.raw_full[i % kRaw], (i / kRaw) & 1u, kTries);
        } else if (w == 8) {
            // ---- products: Z0 Z1 | O0(0) Z0(2) | O1(1) Z1(3) | ...
            const uint32_t id_z = tc::idesc_bf16(128, kRows) & ~((1u << 7) | (1u << 10));  // f16 operands
            const uint32_t id_o = id_z | (1u << 15) | (1u << 16);                          // both with K outermost
            const uint32_t qa = tc::smem_u32(sq), ka = tc::smem_u32(sk), va = tc::smem_u32(sv), pa = tc::smem_u32(sp);
            uint32_t kc = 0, vc = 0, qc = 0, pc[2] = {0, 0};
            bool ok = true;
            auto issue_z = [&](int st) {
                if (!warp_wait(&sh.k_ready[kc & 1], (kc >> 1) & 1u)) return false;
                tc::fence_after_sync();
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint32_t step = (x & 3) * 32;
                    mma_ss(tm + kRows * st, desc_qk(ka + (kc & 1) * kTileBytes + (x >> 2) * kColBlk + step), desc_qk(qa + (x >> 2) * kQBlk + step), id_z, x > 0);
                }
                commit(&sh.z_full[st]);
                commit(&sh.k_free[kc & 1]);
                ++kc;
                return true;
            };
            while (ok && walk.next(a, row_tiles, s)) {
                ok = warp_wait(&sh.q_ready, qc++ & 1u) && issue_z(0);
                if (ok && s.count > 1) ok = issue_z(1);
                for (int i = 0; i < s.count && ok; ++i, ++vc) {
                    const int st = i & 1;
                    ok = warp_wait(&sh.v_ready[vc & 1], (vc >> 1) & 1u) &&
                         warp_wait(&sh.p_full[st], (st ? pc[1]++ : pc[0]++) & 1u);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t v = va + (vc & 1) * kTileBytes;
#pragma unroll
                    for (int x = 0; x < kBlk / 16; ++x)
                        mma_vp(tm + 2 * kRows + kRows * st, desc_v(v + x * 2048, kColBlk), pa + st * kPBytes + x * 1024, id_o, i > 1 || x > 0);
                    commit(&sh.v_free[vc & 1]);
                    if (i + 2 < s.count) ok = issue_z(st);  // its commit also covers O's product
                    else commit(&sh.o_full[st]);
                }
            }
            if (!ok || *dead != 0u) {
                *dead = 1u;
                commit(&sh.drained);  // products in flight end before tensor memory is given back
                (void)warp_wait(&sh.drained, 0);
            }
        } else {
            // ---- conversion: 16 codes a thread at a time, into the products' layout
            const int me = tid - 10 * 32;
            constexpr int RC = D / 16;  // 16-code pieces of a row
            uint32_t blk = 0, turn = 0;
            bool ok = true;
            for (; ok && walk.next(a, row_tiles, s); ++turn) {
                for (int i = s.i0; i < s.i0 + s.count && ok; ++i, ++blk) {
                    const int key0 = i * kBlk;
#pragma unroll 1
                    for (int x = 0; x < 2 && ok; ++x) {
                        const uint32_t it = 2 * blk + x, st = it % kRaw;
                        ok = warp_wait(x ? &sh.v_free[blk & 1] : &sh.k_free[blk & 1], ((blk >> 1) & 1u) ^ 1u) &&
                             warp_wait(&sh.raw_full[st], (it / kRaw) & 1u);
                        if (!ok) break;
                        const unsigned char* src = raw + st * kRawBytes;
                        unsigned char* dst = (x ? sv : sk) + (blk & 1) * kTileBytes;
                        const uint32_t there = sh.has[blk & 7];
                        const bool edge = x && (key0 + kBlk > s.len - a.L + 1 || there != 0xffu);
                        constexpr int kTurns = (kBlk * RC + kConvert - 1) / kConvert;
                        // Sixteen lanes take two rows, eight of them half of each: what they read then fills
                        // the banks once, and so do their 16-byte stores, which the layout puts at
                        // even places of one row and odd places of the other.
                        auto row_of = [](int p) { return 2 * (p >> 4) + ((p >> 2) & 1); };
                        auto piece_of = [](int p) { return (p & 3) + 4 * (((p >> 2) ^ (p >> 3)) & 1); };
                        static_assert(RC == 8, "eight pieces a row");
                        auto store = [&](int p, const uint32_t (&c)[4]) {
                            const int row = row_of(p), ch = piece_of(p);
                            uint32_t h[8];
#pragma unroll
                            for (int q = 0; q < 4; ++q) widen<kE4m3>(c[q], h[2 * q], h[2 * q + 1]);
                            unsigned char* at = dst + (ch >> 2) * kColBlk + row * 128;
                            const int cc = (2 * ch) & 7;
                            *reinterpret_cast<uint4*>(at + ((cc ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4*>(at + (((cc + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
                        };
                        if (!edge) {
                            uint4 u[kTurns];
#pragma unroll
                            for (int e = 0; e < kTurns; ++e) {
                                const int p = me + e * kConvert;
                                if (p < kBlk * RC) u[e] = *reinterpret_cast<const uint4*>(src + row_of(p) * D + piece_of(p) * 16);
                            }
#pragma unroll
                            for (int e = 0; e < kTurns; ++e) {
                                const int p = me + e * kConvert;
                                const uint32_t c[4] = {u[e].x, u[e].y, u[e].z, u[e].w};
                                if (p < kBlk * RC) store(p, c);
                            }
                        } else {
                            // keys that are not there, and NaN that not every row may see, leave the tile
                            for (int p = me; p < kBlk * RC; p += kConvert) {
                                const int row = row_of(p), ch = piece_of(p);
                                const uint4 u = *reinterpret_cast<const uint4*>(src + row * D + ch * 16);
                                uint32_t c[4] = {u.x, u.y, u.z, u.w};
                                const bool is = key0 + row < s.len && ((there >> (row >> 4)) & 1u) != 0u;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    if (!is) c[q] = 0u;
                                    if constexpr (kE4m3) {
                                        const uint32_t nan = __vcmpeq4(c[q] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                        if (nan != 0u) {
                                            for (int y = 0; y < 4; ++y)
                                                if ((nan >> (8 * y)) & 1u)
                                                    atomicMin(&sh.odd[turn & 3][ch * 16 + q * 4 + y], odd_note(turn, key0 + row, s.len - a.L));
                                            c[q] &= ~nan;
                                        }
                                    }
                                }
                                store(p, c);
                            }
                        }
                        tc::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tc::mbar_arrive(x ? &sh.v_ready[blk & 1] : &sh.k_ready[blk & 1]);
                            tc::mbar_arrive(&sh.raw_free[st]);
                        }
                    }
                }
            }
            if (!ok) *dead = 1u;
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax: stream st takes the segment's blocks st, st + 2, ..., a thread the key of its lane
        const int st = w >> 2, q4 = w & 3, key_in = tid & 127;
        const uint32_t lanes = (uint32_t)q4 << 21;
        const uint32_t zt = tm + kRows * st + lanes, ot = tm + 2 * kRows + kRows * st + lanes;
        uint32_t zc = 0, oc = 0, qc = 0, blk0 = 0, turn = 0, jc = 0;
        float* po = reinterpret_cast<float*>(a.ws + L.o);
        float2* ml = reinterpret_cast<float2*>(a.ws + L.ml);
        const float unit_scale = 0.0078125f * a.scale * kLog2e;  // 2^-7 (see row_unit)
        auto larger = [](float x, float y) { return fmaxf(x, y); };
        auto added = [](float x, float y) { return x + y; };
        bool gone = false;
        for (; !gone && walk.next(a, row_tiles, s); ++turn) {
            const int row0 = s.rt * kRows, rows = min(kRows, rows_all - row0);
            const int whole_seen = s.len - a.L;  // keys before this one are seen by every row
            if (st == 0) {
                // the rows of q, each scaled by a power of two, into the products' layout: thread (row, quarter)
                const bool late = turn > 0 && !warp_wait(&sh.f_read, (turn - 1) & 1u);  // the other stream has the last factor
                const int r = key_in >> 2, quarter = key_in & 3;
                const int R = row0 + r, t = R / a.group, head = s.h * a.group + (R - t * a.group);
                const bool on = r < rows;
                uint4 u[4];
                const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)s.n * a.L + t) * a.qs + (int64_t)head * D;
#pragma unroll
                for (int c = 0; c < 4; ++c) u[c] = on ? __ldg(reinterpret_cast<const uint4*>(q) + 4 * quarter + c) : make_uint4(0u, 0u, 0u, 0u);
                if (quarter == 0 && on) sh.at[r] = ((int64_t)s.n * a.L + t) * tokrow + (int64_t)head * D;
                uint32_t top = 0u;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    top = __vmaxu2(__vmaxu2(top, u[c].x & 0x7fff7fffu), __vmaxu2(u[c].y & 0x7fff7fffu, __vmaxu2(u[c].z & 0x7fff7fffu, u[c].w & 0x7fff7fffu)));
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));  // the row's four threads
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int unit = row_unit(top);
                const bool some = any4(0, unit != 0);
                gone = late;  // made the same for all below
                const float up = __uint_as_float((uint32_t)(127 + 7 - unit) << 23);
                auto cv = [&](uint32_t x) { return pack_f16(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up); };
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int ch = 4 * quarter + c;
                    *reinterpret_cast<uint4*>(sq + (ch >> 3) * kQBlk + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                        make_uint4(cv(u[c].x), cv(u[c].y), cv(u[c].z), cv(u[c].w));
                }
                if (quarter == 0) sh.f[r] = __uint_as_float((uint32_t)(127 + unit) << 23);
                if (key_in == 0) sh.mixed = some;
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.q_ready);
            }
            const bool no_q = !warp_wait(&sh.q_ready, qc++ & 1u);
            const bool mixed = sh.mixed != 0u;
            gone = any4(st, no_q || gone);
            if (st == 1 && lane == 0) tc::mbar_arrive(&sh.f_read);
            float l[kRows], vu = 0.f, vtop = 0.f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) l[r] = 0.f;
            if (key_in < kRows) sh.ref[st][key_in] = -FLT_MAX;  // finite: a score of -inf then weighs nothing
            (void)any4(st, false);
            // (two copies: with the rows' own units in the one that runs, ordinary blocks took 3 to 7 % longer)
            auto blocks = [&](auto own) {
                constexpr bool kOwn = decltype(own)::value;
                for (int i = st; i < s.count && !gone; i += 2) {
                    const bool late = !warp_wait(&sh.z_full[st], zc++ & 1u);
                    tc::fence_after_sync();
                    const int b = (int)((blk0 + i) & 7u), key = (s.i0 + i) * kBlk + key_in;
                    uint32_t z[kRows];
                    tmem_ld32(zt, z);
                    const float ks = sh.ks[b][key_in >> 4], vs = sh.vs[b][key_in >> 4];
                    const bool is = key < s.len && ((sh.has[b] >> (key_in >> 4)) & 1u) != 0u;
                    // rows [from, 32) see this key: later tokens of the window see more
                    const int from = !is ? kRows : key < whole_seen ? 0 : max(0, (key - whole_seen) * a.group - row0);
                    float big = 0.f;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const float v = fabsf(sh.vs[b][g]);
                        if (v < INFINITY) big = fmaxf(big, v);
                    }
                    const bool unit = !(big <= vu && big * 64.f >= vu) && big > 0.f;  // the same for every thread
                    const float sc = unit_scale * ks;
                    // Scores less their rows' references; does any pass 2^15 (the largest had 2^7 when its reference was set)?
                    // Where rows have units of their own, or scores may pass 2^20 (|z| < 2^31), this is not yet the answer.
                    const bool far = fabsf(sc) > kFar;
                    float over = -INFINITY;
                    auto less_ref = [&](float mul) {
#pragma unroll
                        for (int c = 0; c < kRows / 4; ++c) {
                            const float4 m = *reinterpret_cast<const float4*>(&sh.ref[st][4 * c]);
                            z[4 * c] = __float_as_uint(fmaf(f_of(z[4 * c]), mul, -m.x));
                            z[4 * c + 1] = __float_as_uint(fmaf(f_of(z[4 * c + 1]), mul, -m.y));
                            z[4 * c + 2] = __float_as_uint(fmaf(f_of(z[4 * c + 2]), mul, -m.z));
                            z[4 * c + 3] = __float_as_uint(fmaf(f_of(z[4 * c + 3]), mul, -m.w));
                        }
                    };
                    tc::tmem_wait_ld();
                    less_ref(sc);
                    if (from == 0) {
#pragma unroll
                        for (int r = 0; r < kRows; r += 2) over = max3(over, f_of(z[r]), f_of(z[r + 1]));
                    } else {
#pragma unroll
                        for (int r = 0; r < kRows; ++r)
                            if (r >= from) over = fmaxf(over, f_of(z[r]));
                    }
                    if (any4(st, over > 15.f || unit || late || kOwn || far)) {
                        gone = any4(st, late);
                        if (gone) break;
                        // new references: the largest scores met so far
                        {
                            float x[kRows];
                            tmem_ld32(zt, reinterpret_cast<uint32_t*>(x));
                            tc::tmem_wait_ld();
                            if constexpr (kOwn) {
#pragma unroll
                                for (int r = 0; r < kRows; ++r) x[r] *= sh.f[r];
                            }
#pragma unroll
                            for (int r = 0; r < kRows; ++r) x[r] = r >= from ? x[r] * sc : -INFINITY;
                            sh.top[st][q4][lane] = reduce_rows(x, larger);
                        }
                        (void)any4(st, false);
                        float ratio = 1.f;
                        if (unit) {
                            vtop = fmaxf(vtop, big);
                            const float nu = fmaxf(big, vtop * 9.094947e-13f);
                            ratio = vu == 0.f ? 0.f : vu / nu;
                            vu = nu;
                        }
                        if (q4 == 0) {
                            const float was = sh.ref[st][lane];
                            const float top = fmaxf(fmaxf(sh.top[st][0][lane], sh.top[st][1][lane]), fmaxf(sh.top[st][2][lane], sh.top[st][3][lane]));
                            const float now = top - was > 15.f ? top - 7.f : was;
                            sh.by[st][lane] = ex2(was - now);
                            sh.ref[st][lane] = now;
                        }
                        (void)any4(st, false);
#pragma unroll
                        for (int r = 0; r < kRows; ++r) l[r] *= sh.by[st][r];
                        if (i >= 2) {
                            // (the products into O up to here ended with the scores that were waited for)
                            uint32_t o[kRows];
                            tmem_ld32(ot, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int r = 0; r < kRows; ++r) o[r] = __float_as_uint(f_of(o[r]) * (sh.by[st][r] * ratio));
                            tmem_st32(ot, o);
                            tc::tmem_wait_st();
                        }
                        // The scores anew, in the rows' units.  Large ones are rounded, as their reference was, before it comes off,
                        // so that none passes the largest, however large they are.
                        tmem_ld32(zt, z);
                        tc::tmem_wait_ld();
                        if constexpr (kOwn) {
#pragma unroll
                            for (int r = 0; r < kRows; ++r) {
                                const float x = f_of(z[r]) * sh.f[r], m = sh.ref[st][r];
                                z[r] = __float_as_uint(sh.f[r] * fabsf(sc) > kFar ? __fmul_rn(x, sc) - m : fmaf(x, sc, -m));
                            }
                        } else {
                            const float mul = far ? 1.f : sc, up = far ? sc : 1.f;
#pragma unroll
                            for (int r = 0; r < kRows; ++r) z[r] = __float_as_uint(__fmul_rn(f_of(z[r]), up));
                            less_ref(mul);
                        }
                    }
                    const float pv = vu == 0.f ? (vs == vs ? 0.f : vs) : vs / vu;
                    unsigned char* at = sp + st * kPBytes + key_in * 64;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 8 * c + 2 * e;
                            // a row that has seen nothing has the first reference; its weights are replaced below
                            float2 y = make_float2(ex2(f_of(z[r])), ex2(f_of(z[r + 1])));
                            if (from > 0) {
                                if (r < from) y.x = 0.f;
                                if (r + 1 < from) y.y = 0.f;
                            }
                            l[r] += y.x;
                            l[r + 1] += y.y;
                            y = __fmul2_rn(y, make_float2(pv, pv));
                            p[e] = pack_f16(y.x, y.y);
                        }
                        *reinterpret_cast<uint4*>(at + ((c ^ ((key_in >> 1) & 3)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    tc::fence_async_smem();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sh.p_full[st]);
                }
            };
            if (mixed) blocks(std::true_type{});
            else blocks(std::false_type{});
            blk0 += s.count;
            const bool both = s.count > 1;
            bool late = false;
            if (!gone && st < s.count) late = !warp_wait(&sh.o_full[st], oc++ & 1u);
            gone = any4(st, late || gone);
            tc::fence_after_sync();
            if (gone) break;
            // a row's sum over the keys, by warp; the reference and the unit
            sh.sum[st][q4][lane] = reduce_rows(l, added);
            if (q4 == 0 && lane == 0) sh.unit[st] = vu;
            __syncwarp();
            if (st == 1) {
                if (both) {
                    if (lane == 0) tc::mbar_arrive(&sh.joined);
                    late = !warp_wait(&sh.join_free, jc++ & 1u);
                }
                gone = any4(1, late);
                continue;
            }
            if (both) late = !warp_wait(&sh.joined, jc++ & 1u);
            gone = any4(0, late);
            if (gone) break;
            const bool whole = s.begun && s.ended;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (s.begun ? 1 : 0);
            if (q4 == 0) {  // lane r: row r's weights of the two streams
                const float m0 = sh.ref[0][lane], m1 = both ? sh.ref[1][lane] : -FLT_MAX;
                const float l0 = (sh.sum[0][0][lane] + sh.sum[0][1][lane]) + (sh.sum[0][2][lane] + sh.sum[0][3][lane]);
                const float l1 = both ? (sh.sum[1][0][lane] + sh.sum[1][1][lane]) + (sh.sum[1][2][lane] + sh.sum[1][3][lane]) : 0.f;
                const float mm = fmaxf(m0, m1);
                const float f0 = ex2(m0 - mm), f1 = ex2(m1 - mm);
                const float sum = l0 * f0 + l1 * f1;
                const float mul = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                sh.weight[0][lane] = sh.unit[0] * f0 * mul;
                sh.weight[1][lane] = both ? sh.unit[1] * f1 * mul : 0.f;
                if (!whole && lane < rows) ml[slot * rows_max + lane] = make_float2(mm, sum);
            }
            (void)any4(0, false);
            uint32_t o[kRows], y[kRows];
            tmem_ld32(ot, o);
            if (both) tmem_ld32(ot + kRows, y);
            tc::tmem_wait_ld();
            // a NaN in this thread's channel reaches the rows that see its key
            int nan_from = kRows;
            if (kE4m3) {
                const unsigned long long od = sh.odd[turn & 3][key_in];
                if ((uint32_t)(od >> 32) == 0xfffffffeu - turn) nan_from = (int)max((int64_t)0, min((int64_t)kRows, (int64_t)(uint32_t)od * a.group - row0));
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float x = f_of(o[r]) * sh.weight[0][r];
                if (both) x = fmaf(f_of(y[r]), sh.weight[1][r], x);
                if (r >= nan_from) x = NAN;
                if (r < rows) {
                    if (whole) static_cast<__nv_bfloat16*>(a.out)[sh.at[r] + key_in] = __float2bfloat16_rn(x);
                    else po[(slot * rows_max + r) * D + key_in] = x;
                }
            }
            tc::fence_before_sync();
            (void)any4(0, false);  // sh.weight and sh.at are read
            if (both && lane == 0) tc::mbar_arrive(&sh.join_free);
        }
        if (gone) *dead = 1u;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (w == 8) tc::tmem_dealloc(tm, 128);
    if (tid == 0) {
        // what this worker leaves to be joined: the unit that it began and did not end
        Record mine{-1, 0, 0, 0, 0};
        const bool failed = sh.dead != 0u;
        walk.left = sh.left;
        walk.gap = gap;
        walk.c = sh.begin;
        int64_t pos = b1 - sh.left;
        while (walk.next(a, row_tiles, s)) {
            if (s.begun) {
                Record rec{-1, 0, 0, 0, 0};
                if (!s.ended && !failed) {
                    const int64_t e = pos + tiles_of<kBlk>(s.len);  // past the unit's last block
                    rec = Record{s.n, s.h, s.rt, (int32_t)blockIdx.x, (int32_t)((e * W + total - 1) / total - 1)};
                    mine = rec;
                }
                if (by_unit) records[unit_of(s)] = rec;
            }
            pos += s.count + gap;
        }
        if (!by_unit) records[blockIdx.x] = mine;
        reinterpret_cast<uint32_t*>(a.ws + L.flags)[blockIdx.x] = sh.flag | (failed ? kCheckTimeout : 0u);
    }
}

namespace {

template <bool kE4m3>
cudaError_t launch_window_d(const AttnDecodeArgs& a, cudaStream_t s)
{
    static_assert(kSmem + sizeof(Shared) <= 232448, "the tiles fit an SM");
    static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= kThreads * 128, "register split");
    auto kern = kda_attn_window_kernel<kE4m3>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, (int)kSmem);
    if (e != cudaSuccess) return e;
    const int64_t rows_all = (int64_t)a.L * a.group;
    const int rows = (int)(rows_all < kRows ? rows_all : kRows);
    const int64_t units = (int64_t)a.N * a.Hkv * ((rows_all + kRows - 1) / kRows);
    const double most = (double)units * (((int64_t)a.c.max_pages * a.c.page + kBlk - 1) / kBlk);
    const int full = sm_count_of_current_device();
    const int ctas = most < (double)full ? (int)most : full;
    const bool by_unit = units <= ctas;
    kern<<<ctas, kThreads, kSmem, s>>>(a, rows, by_unit);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_attn_join(a, KDA_BF16, rows, kRows, ctas, ctas, by_unit, units, s);
}

}  // namespace

// From 25 rows a key head, where the page table holds more than 512 keys a sequence.  Measured here and on
// the warp-level form, us: 28 rows of 8 heads, 64 sequences of 3150 keys 133 and 193; 56 rows 249 and 365; one
// sequence of 4000, one head 13.8 and 16.1; but 20 rows of one head, 64 of 1000 23.7 and 20.6; and 28 rows of
// 8 heads, 256 of 300 136 and 113, where a unit's start and end outweigh its keys (of 500: 154 and 151, of 700 188 and
// 191).  The lengths are not known here: a table that is wide for its sequences takes this form for short ones too.
bool attn_window_takes(int64_t rows, int d, kda_dtype_t dt, int64_t capacity)
{
    return dt == KDA_BF16 && d == D && rows > 24 && capacity > 512;
}

size_t attn_window_workspace_bytes(int64_t rows, int d)
{
    const int ctas = sm_count_of_current_device();
    return decode_layout(ctas, ctas, (int)(rows < kRows ? rows : kRows), d).total;
}

cudaError_t launch_attn_window(const AttnDecodeArgs& a, cudaStream_t s)
{
    return a.c.dtype == KDA_CACHE_E4M3 ? launch_window_d<true>(a, s) : launch_window_d<false>(a, s);
}

}  // namespace kda
