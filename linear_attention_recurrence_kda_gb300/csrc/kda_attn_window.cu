// kda_attn_window.cu -- many rows a key head over the paged 8-bit cache, on the 5th-generation tensor
// cores (kda_attention_decode: a drafted window, a large group of query heads; bf16, 64 or 128 channels).
//
//   Z = scale ks (Q K^T),  P = 2^(Z - m),  O = sum P V,  o = O / l        as in kda_attn_decode.cu
//
// With 28 rows a key head a warp-level kernel spends about 1300 instructions on a tile of 32 keys, most
// of them conversions and products, and reads the cache at a quarter of HBM's rate.  Here a CTA takes
// up to 128 rows and keys in blocks of 128: the codes are converted once, by warps that do nothing else,
// into f16 tiles (exactly: e4m3 and int8 are subsets of f16) from which tcgen05.mma forms Z and O; a
// block then costs a few hundred instructions a warp.
//
// Blocks alternate between two streams, each with its own maximum, sum and O, so that one stream's
// softmax runs while the other's products do; at the end of a unit the first stream joins them.
// Tensor memory: Z0 | Z1 | O0 | O1, P over the first half of its Z as packed f16.  All units' blocks form
// one line that is cut evenly among the CTAs; pieces of a unit are joined by the join kernel.
//
// Warps 0-3 and 4-7: softmax of the streams (a thread owns a row), 8: products, 9: copies and scales,
// 10-15: conversion.  A row of q enters scaled by a power of two as in kda_attn_decode.cu, V's scales
// through P, with O in units of the block's largest scale.
#include "kda_attn.cuh"
#include "kda_attn_decode.cuh"
#include "kda_attn_tc.cuh"

namespace kda {

using namespace attn;

namespace {

constexpr int kBlk = 128;  // keys per block
constexpr int kRows = 128;
constexpr int kThreads = 512;
constexpr int kConvert = 192;
constexpr int kRaw = 5;    // raw tiles (K and V in turn) on their way or waiting
constexpr int kGroups = kBlk / 16;
// warpgroups' registers after the split: 256 x 168 + 256 x 88 = 512 x 128, what the launch holds
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
constexpr float kLog2e = 1.4426950408889634f;

template <int D> struct Cfg {
    static constexpr int NB = D / 64;
    static constexpr uint32_t BLK = 128 * 128;     // bytes of a 64-channel block of 128 rows
    static constexpr uint32_t TILE = NB * BLK;     // an f16 tile
    static constexpr uint32_t RAW = kBlk * D;      // a tile of codes
    static constexpr uint32_t SMEM = 4 * TILE + kRaw * RAW + 1024;  // Q, K, two of V
};

struct Maps {
    CUtensorMap k, v;
};

struct Shared {
    uint64_t raw_full[kRaw], raw_free[kRaw], k_ready, k_free, v_ready[2], v_free[2];
    uint64_t q_ready, f_read, z_full[2], p_full[2], o_full[2], joined, join_free, drained;
    uint32_t tmem, dead, flag;
    uint32_t has[8];             // by block: bit g, group g of 16 keys is there
    float ks[8][kGroups], vs[8][kGroups];
    float f[kRows];              // what a row's scores are multiplied by
    float part[3][kRows];        // the second stream's maximum, sum and unit
    unsigned long long odd[4][128];  // by the segment's turn: the first key with a NaN in a channel (see odd_note)
    int64_t prefix[kThreads + 1];
};

// A run of a unit's blocks.
struct Segment {
    int n, h, rt, i0, count, len;
    bool begun, ended;  // does it hold the unit's first block, its last?
};

// the segments of a worker, one after the other
struct Walk {
    Cursor c;
    int left;
    __device__ __forceinline__ bool next(const AttnDecodeArgs& a, int row_tiles, Segment& s)
    {
        if (left <= 0) return false;
        s.n = c.n; s.h = c.h; s.rt = c.rt; s.i0 = c.i; s.len = c.len;
        s.count = min(left, c.tiles - c.i);
        s.begun = c.i == 0;
        s.ended = c.i + s.count == c.tiles;
        left -= s.count;
        if (left > 0) {
            c.i = c.tiles - 1;
            next_tile<kBlk>(a, row_tiles, c);
        }
        return true;
    }
};

// A noted NaN: the segment's turn in the upper half (later turns are smaller, so that atomicMin prefers
// them), the key's distance from the last key that every row sees in the lower.  Conversion is at
// most two segments ahead of the softmax, so four arrays in turn never mix.
__device__ __forceinline__ unsigned long long odd_note(uint32_t turn, int key, int last)
{
    return ((unsigned long long)(0xfffffffeu - turn) << 32) | (uint32_t)max(key - last, 0);
}

}  // namespace

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1)
    kda_attn_window_kernel(const AttnDecodeArgs a, const __grid_constant__ Maps maps, const int rows_max, const bool by_unit)
{
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    unsigned char* sq = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sk = sq + C::TILE;
    unsigned char* sv = sk + C::TILE;       // two
    unsigned char* raw = sv + 2 * C::TILE;  // kRaw
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
        tc::mbar_init(&sh.k_ready, kConvert / 32);
        tc::mbar_init(&sh.k_free, 1);
        for (int i = 0; i < 2; ++i) {
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
    if (w == 8) tc::tmem_alloc(&sh.tmem, 512);
    // blocks before every run of `chunk` sequences
    const int chunk = (a.N + kThreads - 1) / kThreads;
    {
        int64_t sum = 0;
        bool bad = false;
        for (int i = 0; i < chunk; ++i) {
            const int n = tid * chunk + i;
            if (n < a.N) sum += tiles_of<kBlk>(length_of(a, n, &bad));
        }
        int64_t x = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        sh.prefix[tid + 1] = x;
        if (tid == 0) sh.prefix[0] = 0;
        __syncthreads();
        if (bad) atomicOr(&sh.flag, kCheckBadSeqlens);
        int64_t before = 0;
        for (int i = 0; i < w; ++i) before += sh.prefix[(i + 1) * 32];
        __syncthreads();
        sh.prefix[tid + 1] = x + before;
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
    const int64_t total = sh.prefix[kThreads] * per_block;
    const int64_t W = min((int64_t)gridDim.x, total);
    const int64_t b0 = blockIdx.x < W ? blockIdx.x * total / W : 0, b1 = blockIdx.x < W ? (blockIdx.x + 1) * total / W : 0;
    Walk walk;
    auto start = [&]() {  // at this CTA's first block: a run of sequences by bisection, then one by one
        walk.left = (int)(b1 - b0);
        walk.c = Cursor{0, 0, 0, 0, 1, 0};
        if (walk.left <= 0) return;
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sh.prefix[mid] * per_block <= b0) lo = mid;
            else hi = mid - 1;
        }
        int64_t at = sh.prefix[lo] * per_block;
        Cursor& c = walk.c;
        c.n = lo * chunk;
        for (;;) {
            c.len = length_of(a, c.n);
            c.tiles = tiles_of<kBlk>(c.len);
            const int64_t here = c.tiles * per_block;
            if (at + here > b0 || c.n + 1 >= a.N) break;
            at += here;
            ++c.n;
        }
        const int64_t rest = b0 - at, unit = rest / c.tiles;
        c.i = (int)(rest - unit * c.tiles);
        c.h = (int)(unit / row_tiles);
        c.rt = (int)(unit - (int64_t)c.h * row_tiles);
    };
    start();
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
                int page = page_of(s, s.i0);
                float scale = scale_of(s, page);
                for (int i = s.i0; i < s.i0 + s.count && ok; ++i, ++blk) {
                    // the next block's page and scale are on their way meanwhile
                    const int page1 = i + 1 < s.i0 + s.count ? page_of(s, i + 1) : -1;
                    const float scale1 = scale_of(s, page1);
                    const uint32_t there = __ballot_sync(0xffffffffu, page >= 0) & 0xffu;
                    if (page == -2) atomicOr(&sh.flag, kCheckBadSeqlens);
                    for (int x = 0; x < 2 && ok; ++x, ++it) {
                        const uint32_t st = it % kRaw;
                        ok = warp_wait(&sh.raw_free[st], ((it / kRaw) & 1u) ^ 1u) && !__any_sync(0xffffffffu, *dead != 0u);
                        if (!ok) break;
                        if (x == 0) {
                            if (lane < 8) sh.ks[blk & 7][grp] = scale;
                            else if (lane < 16) sh.vs[blk & 7][grp] = scale;
                            if (lane == 0) sh.has[blk & 7] = there;
                            __syncwarp();
                        }
                        const int pieces = __popc(there) / gpp + (__popc(there) % gpp != 0 ? 1 : 0);
                        if (lane == 0) tc::mbar_arrive_expect_tx(&sh.raw_full[st], (uint32_t)pieces * box * D);
                        for (int p = 0; p < kGroups / gpp; ++p) {
                            const int id = __shfl_sync(0xffffffffu, page, p * gpp);
                            if (lane == 0 && id >= 0)
                                tc::tma_load_3d(raw + st * C::RAW + p * box * D, x ? &maps.v : &maps.k, 0,
                                                (i * kBlk + p * box) & (a.c.page - 1), id * a.Hkv + s.h, &sh.raw_full[st]);
                        }
                    }
                    page = page1;
                    scale = scale1;
                }
            }
            if (!ok) *dead = 1u;
            if (lane == 0 && *dead)
                for (uint32_t i = it > kRaw ? it - kRaw : 0; i < it; ++i) (void)tc::mbar_wait(&sh.raw_full[i % kRaw], (i / kRaw) & 1u, kTries);
        } else if (w == 8) {
            // ---- products: Z0 Z1 | O0(0) Z0(2) | O1(1) Z1(3) | ...
            const uint32_t id_z = tc::idesc_bf16(128, kBlk) & ~((1u << 7) | (1u << 10));  // f16 operands
            const uint32_t id_o = (tc::idesc_bf16(128, D) & ~((1u << 7) | (1u << 10))) | (1u << 16);
            const uint32_t qa = tc::smem_u32(sq), ka = tc::smem_u32(sk), va = tc::smem_u32(sv);
            uint32_t kc = 0, vc = 0, qc = 0, pc[2] = {0, 0};
            bool ok = true;
            auto issue_z = [&](int st) {
                if (!warp_wait(&sh.k_ready, kc++ & 1u)) return false;
                tc::fence_after_sync();
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint32_t off = (x >> 2) * C::BLK + (x & 3) * 32;
                    mma_ss(tm + 128 * st, desc_qk(qa + off), desc_qk(ka + off), id_z, x > 0);
                }
                commit(&sh.z_full[st]);
                commit(&sh.k_free);
                return true;
            };
            while (ok && walk.next(a, row_tiles, s)) {
                ok = warp_wait(&sh.q_ready, qc++ & 1u) && issue_z(0);
                if (ok && s.count > 1) ok = issue_z(1);
                for (int i = 0; i < s.count && ok; ++i, ++vc) {
                    const int st = i & 1;
                    ok = warp_wait(&sh.v_ready[vc & 1], (vc >> 1) & 1u) &&
                         warp_wait(&sh.p_full[st], (st ? pc[1]++ : pc[0]++) & 1u) && !__any_sync(0xffffffffu, *dead != 0u);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t v = va + (vc & 1) * C::TILE;
#pragma unroll
                    for (int x = 0; x < kBlk / 16; ++x)
                        mma_ts(tm + 256 + D * st, tm + 128 * st + 8 * x, desc_v(v + x * 2048, D == 128 ? C::BLK : 1024u), id_o,
                               i > 1 || x > 0);
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
            uint32_t it = 0, kc = 0, vc = 0, blk = 0, turn = 0;
            bool ok = true;
            for (; ok && walk.next(a, row_tiles, s); ++turn) {
                for (int i = s.i0; i < s.i0 + s.count && ok; ++i, ++blk, ++vc, ++kc) {
                    const int key0 = i * kBlk;
                    for (int x = 0; x < 2 && ok; ++x, ++it) {
                        const uint32_t st = it % kRaw;
                        ok = warp_wait(&sh.raw_full[st], (it / kRaw) & 1u) &&
                             (x ? warp_wait(&sh.v_free[vc & 1], ((vc >> 1) & 1u) ^ 1u) : warp_wait(&sh.k_free, (kc & 1u) ^ 1u)) &&
                             !__any_sync(0xffffffffu, *dead != 0u);
                        if (!ok) break;
                        const unsigned char* src = raw + st * C::RAW;
                        unsigned char* dst = x ? sv + (vc & 1) * C::TILE : sk;
                        const uint32_t there = sh.has[blk & 7];
                        const bool edge = x && (key0 + kBlk > s.len - a.L + 1 || there != 0xffu);
#pragma unroll 2
                        for (int e = 0; e < (kBlk * RC + kConvert - 1) / kConvert; ++e) {
                            const int p = me + e * kConvert, row = p / RC, ch = p % RC;
                            if (p >= kBlk * RC) break;
                            const uint4 u = *reinterpret_cast<const uint4*>(src + p * 16);
                            uint32_t c[4] = {u.x, u.y, u.z, u.w};
                            if (edge) {
                                // keys that are not there, and NaN that not every row may see, leave the tile
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
                            }
                            uint32_t h[8];
#pragma unroll
                            for (int q = 0; q < 4; ++q) widen<kE4m3>(c[q], h[2 * q], h[2 * q + 1]);
                            unsigned char* at = dst + (ch >> 2) * C::BLK + row * 128;
                            const int cc = (2 * ch) & 7;
                            *reinterpret_cast<uint4*>(at + ((cc ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4*>(at + (((cc + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                        tc::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tc::mbar_arrive(x ? &sh.v_ready[vc & 1] : &sh.k_ready);
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
        // ---- softmax: stream st takes the segment's blocks st, st + 2, ..., a thread the row of its lane
        const int st = w >> 2, r = tid & 127, q4 = w & 3;
        const uint32_t lanes = (uint32_t)q4 << 21;
        const uint32_t zt = tm + 128 * st + lanes, ot = tm + 256 + D * st + lanes;
        uint32_t zc = 0, oc = 0, qc = 0, blk0 = 0, turn = 0, jc = 0;
        float* po = reinterpret_cast<float*>(a.ws + L.o);
        float2* ml = reinterpret_cast<float2*>(a.ws + L.ml);
        bool gone = false;
        for (; !gone && walk.next(a, row_tiles, s); ++turn) {
            const int R = s.rt * kRows + r;
            const bool on = R < rows_all;
            const bool warp_on = s.rt * kRows + 32 * q4 < rows_all;
            const int t = on ? R / a.group : 0, head = s.h * a.group + (on ? R - t * a.group : 0);
            const int seen = on ? s.len - a.L + t + 1 : 0;
            float f = 0.f;
            if (st == 0) {
                // (the other stream has the last segment's factors)
                if (turn > 0 && !warp_wait(&sh.f_read, (turn - 1) & 1u)) gone = true;
                // the row of q, scaled so that its largest value lies in [2^14, 2^15), into the products' layout
                if (on) {
                    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)s.n * a.L + t) * a.qs +
                                                                    (int64_t)head * D);
                    uint32_t top = 0u;
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 u = __ldg(q + c);
                        top = __vmaxu2(__vmaxu2(top, u.x & 0x7fff7fffu), __vmaxu2(u.y & 0x7fff7fffu, __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
                    }
                    int e = (int)(max(top & 0xffffu, top >> 16) >> 7) - 127;
                    e = min(max(e, -100), 127);
                    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
                    f = __uint_as_float((uint32_t)(127 + e - 14) << 23) * a.scale * kLog2e;
                    auto cv = [&](uint32_t x) { return pack_f16(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up); };
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 u = __ldg(q + c);
                        *reinterpret_cast<uint4*>(sq + (c >> 3) * C::BLK + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                            make_uint4(cv(u.x), cv(u.y), cv(u.z), cv(u.w));
                    }
                }
                sh.f[r] = f;
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.q_ready);
            } else {
                if (!warp_wait(&sh.q_ready, qc & 1u)) gone = true;
                f = sh.f[r];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.f_read);
            }
            ++qc;
            float m = -INFINITY, l = 0.f, vu = 0.f, vtop = 0.f;
            for (int i = st; i < s.count && !gone; i += 2) {
                gone = !warp_wait(&sh.z_full[st], zc++ & 1u) || __any_sync(0xffffffffu, *dead != 0u);
                if (gone) break;
                tc::fence_after_sync();
                if (warp_on) {
                    const int b = (int)((blk0 + i) & 7u), key0 = (s.i0 + i) * kBlk;
                    const uint32_t there = sh.has[b];
                    const bool edge = key0 + kBlk > s.len - a.L + 1 || there != 0xffu;
                    // bit c: key key0 + c of this half is seen
                    auto seen_of = [&](int half) -> uint64_t {
                        uint64_t x = 0;
                        const int k = seen - key0 - 64 * half;
                        x = k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1ull;
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            if (!((there >> (4 * half + g)) & 1u)) x &= ~(0xffffull << (16 * g));
                        return x;
                    };
                    float top = -INFINITY;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t z[64];
                        tmem_ld32(zt + 64 * half, z);
                        tmem_ld32(zt + 64 * half + 32, z + 32);
                        tc::tmem_wait_ld();
                        if (edge) {
                            const uint64_t vis = seen_of(half);
#pragma unroll
                            for (int c = 0; c < 64; ++c)
                                if ((vis >> c) & 1ull) top = fmaxf(top, f_of(z[c]) * (f * sh.ks[b][4 * half + (c >> 4)]));
                        } else {
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const float sg = f * sh.ks[b][4 * half + g];
                                float x = -INFINITY, y = -INFINITY;
#pragma unroll
                                for (int c = 16 * g; c < 16 * g + 16; c += 4) {
                                    x = max3(x, f_of(z[c]) * sg, f_of(z[c + 1]) * sg);
                                    y = max3(y, f_of(z[c + 2]) * sg, f_of(z[c + 3]) * sg);
                                }
                                top = max3(top, x, y);
                            }
                        }
                    }
                    // the reference and O's unit (the same for all rows), and O where either has moved
                    const float now = top > m + 8.f ? top : m;
                    const float ref = now == -INFINITY ? 0.f : now;
                    float by = ex2(m - ref);
                    bool moved = now != m;
                    m = now;
                    l *= by;
                    float big = 0.f;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const float v = fabsf(sh.vs[b][g]);
                        if (v < INFINITY) big = fmaxf(big, v);
                    }
                    if (!(big <= vu && big * 64.f >= vu) && big > 0.f) {
                        vtop = fmaxf(vtop, big);
                        const float nu = fmaxf(big, vtop * 9.094947e-13f);
                        by *= vu == 0.f ? 0.f : vu / nu;
                        vu = nu;
                        moved = true;
                    }
                    if (i >= 2 && __any_sync(0xffffffffu, moved)) {
                        // the products into O up to here ended with the scores that were waited for
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(ot + 32 * c, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(f_of(o[e]) * by);
                            tmem_st32(ot + 32 * c, o);
                        }
                    }
                    const float iv = vu == 0.f ? 0.f : 1.f / vu;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t z[64];
                        // (P lies over Z's first half: the second is read before P's second part is written there)
                        tmem_ld32(zt + 64 * half, z);
                        tmem_ld32(zt + 64 * half + 32, z + 32);
                        tc::tmem_wait_ld();
                        const uint64_t vis = edge ? seen_of(half) : ~0ull;
                        uint32_t p[32];
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const float sg = f * sh.ks[b][4 * half + g];
                            const float vs = sh.vs[b][4 * half + g];
                            const float pv = vu == 0.f ? (vs == vs ? 0.f : vs) : vs * iv;
                            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                            for (int c = 16 * g; c < 16 * g + 16; c += 2) {
                                const float2 x = __ffma2_rn(make_float2(f_of(z[c]), f_of(z[c + 1])), make_float2(sg, sg), make_float2(-ref, -ref));
                                float2 y = make_float2(ex2(x.x), ex2(x.y));
                                if (edge) {
                                    if (!((vis >> c) & 1ull)) y.x = 0.f;
                                    if (!((vis >> (c + 1)) & 1ull)) y.y = 0.f;
                                }
                                sum = __fadd2_rn(sum, y);
                                y = __fmul2_rn(y, make_float2(pv, pv));
                                p[c >> 1] = pack_f16(y.x, y.y);
                            }
                            l += sum.x + sum.y;
                        }
                        tmem_st32(zt + 32 * half, p);
                    }
                    tc::tmem_wait_st();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.p_full[st]);
            }
            blk0 += s.count;
            const bool both = s.count > 1;
            if (!gone && st < s.count) gone = !warp_wait(&sh.o_full[st], oc++ & 1u) || __any_sync(0xffffffffu, *dead != 0u);
            tc::fence_after_sync();
            if (both && !gone) {
                if (st == 1) {
                    sh.part[0][r] = m;
                    sh.part[1][r] = l;
                    sh.part[2][r] = vu;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sh.joined);
                    gone = !warp_wait(&sh.join_free, jc++ & 1u);
                } else {
                    gone = !warp_wait(&sh.joined, jc++ & 1u);
                }
            }
            if (st == 0 && !gone) {
                const float m1 = both ? sh.part[0][r] : -INFINITY, l1 = both ? sh.part[1][r] : 0.f, u1 = both ? sh.part[2][r] : 0.f;
                const float mm = fmaxf(m, m1), ref = mm == -INFINITY ? 0.f : mm;
                const float f0 = ex2(m - ref), f1 = ex2(m1 - ref);
                const float sum = l * f0 + l1 * f1;
                const bool whole = s.begun && s.ended;
                const float mul = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                const float w0 = vu * f0 * mul, w1 = u1 * f1 * mul;
                const int64_t slot = 2 * (int64_t)blockIdx.x + (s.begun ? 1 : 0);
                if (warp_on) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32], y[32];
                        tmem_ld32(ot + 32 * c, o);
                        if (both) tmem_ld32(ot + D + 32 * c, y);
                        tc::tmem_wait_ld();
                        float x[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            x[e] = f_of(o[e]) * w0 + (both ? f_of(y[e]) * w1 : 0.f);
                            if (kE4m3) {
                                const unsigned long long od = sh.odd[turn & 3][32 * c + e];
                                if ((uint32_t)(od >> 32) == 0xfffffffeu - turn && (int64_t)(uint32_t)od + s.len - a.L < seen) x[e] = NAN;
                            }
                        }
                        if (!on) continue;
                        if (whole) {
                            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)s.n * a.L + t) * tokrow + (int64_t)head * D + 32 * c;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                *reinterpret_cast<uint4*>(out + 8 * e) = make_uint4(tc::pack_bf16(x[8 * e], x[8 * e + 1]), tc::pack_bf16(x[8 * e + 2], x[8 * e + 3]),
                                                                                   tc::pack_bf16(x[8 * e + 4], x[8 * e + 5]), tc::pack_bf16(x[8 * e + 6], x[8 * e + 7]));
                        } else {
                            float* pd = po + (slot * rows_max + r) * D + 32 * c;
#pragma unroll
                            for (int e = 0; e < 8; ++e) *reinterpret_cast<float4*>(pd + 4 * e) = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                        }
                    }
                    if (on && !whole) ml[slot * rows_max + r] = make_float2(mm, sum);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (both && lane == 0) tc::mbar_arrive(&sh.join_free);
            }
        }
        if (gone) *dead = 1u;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (w == 8) tc::tmem_dealloc(tm, 512);
    if (tid == 0) {
        // what this worker leaves to be joined: the unit that it began and did not end
        Record mine{-1, 0, 0, 0, 0};
        const bool failed = sh.dead != 0u;
        start();
        int64_t pos = b0;
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
            pos += s.count;
        }
        if (!by_unit) records[blockIdx.x] = mine;
        reinterpret_cast<uint32_t*>(a.ws + L.flags)[blockIdx.x] = sh.flag | (failed ? kCheckTimeout : 0u);
    }
}

namespace {

bool encode_codes(CUtensorMap* m, const void* base, const AttnDecodeArgs& a)
{
    const TensorMapEncode enc = attn_tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.c.page, (cuuint64_t)a.c.num_pages * a.Hkv};
    const cuuint64_t strides[2] = {(cuuint64_t)a.d, (cuuint64_t)a.d * a.c.page};
    const cuuint32_t box[3] = {(cuuint32_t)a.d, (cuuint32_t)(a.c.page < kBlk ? a.c.page : kBlk), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kE4m3>
cudaError_t launch_window_d(const AttnDecodeArgs& a, cudaStream_t s)
{
    static_assert(Cfg<D>::SMEM + sizeof(Shared) <= 232448, "the tiles fit an SM");
    static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= kThreads * 128, "register split");
    Maps maps;
    if (!encode_codes(&maps.k, a.c.k, a) || !encode_codes(&maps.v, a.c.v, a)) return cudaErrorInvalidValue;
    auto kern = kda_attn_window_kernel<D, kE4m3>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, (int)Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t rows_all = (int64_t)a.L * a.group;
    const int rows = (int)(rows_all < kRows ? rows_all : kRows);
    const int64_t units = (int64_t)a.N * a.Hkv * ((rows_all + kRows - 1) / kRows);
    const double most = (double)units * (((int64_t)a.c.max_pages * a.c.page + kBlk - 1) / kBlk);
    const int full = sm_count_of_current_device();
    const int ctas = most < (double)full ? (int)most : full;
    const bool by_unit = units <= ctas;
    kern<<<ctas, kThreads, Cfg<D>::SMEM, s>>>(a, maps, rows, by_unit);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_attn_join(a, KDA_BF16, rows, kRows, ctas, ctas, by_unit, units, s);
}

}  // namespace

bool attn_window_takes(int64_t rows, int d, kda_dtype_t dt) { return dt == KDA_BF16 && d != 32 && rows > 16; }

size_t attn_window_workspace_bytes(int64_t rows, int d)
{
    const int ctas = sm_count_of_current_device();
    return decode_layout(ctas, ctas, (int)(rows < kRows ? rows : kRows), d).total;
}

cudaError_t launch_attn_window(const AttnDecodeArgs& a, cudaStream_t s)
{
    const bool e4m3 = a.c.dtype == KDA_CACHE_E4M3;
    if (a.d == 64) return e4m3 ? launch_window_d<64, true>(a, s) : launch_window_d<64, false>(a, s);
    return e4m3 ? launch_window_d<128, true>(a, s) : launch_window_d<128, false>(a, s);
}

}  // namespace kda
