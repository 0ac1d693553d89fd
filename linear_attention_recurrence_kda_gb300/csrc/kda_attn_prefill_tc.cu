// kda_attn_prefill_tc.cu -- causal attention over packed prompts on the 5th-generation tensor cores:
// bf16 (kda_attention_prefill).
//
//   Z = scale Q K^T,  P = 2^(Z log2 e - m),  O = sum P V,  o = O / l      per row, keys in tiles of 128
//
// A CTA holds two halves of 128 rows (the query heads of a group times 128 / group tokens each, so
// that a group shares every K and V tile) and walks the keys of both.  Products are tcgen05.mma with
// M = 128: Z from Q and K in shared memory, O += P V with P read from tensor memory and V taken
// token-major as it lies in shared memory.  Tensor memory: Z0 | Z1 | O0 | O1 (128 columns each at 128
// channels), P over the first half of its Z as packed bf16.  Up to 64 channels leave room for P0 | P1:
// the next Z is then formed while the softmax is at work on the last one.
//
// The tensor cores are the bound: 4 x 128 x 128 x 128 multiply-adds per key tile and CTA, 2048 cycles
// at 4096 a cycle, against 1024 cycles of exponentials (32 a cycle) and about 800 of issue.  So the
// roles are split by warp and meet only at mbarriers: while one half's products run, the other
// half's softmax does.  Warps 0-3 and 4-7 own the halves (a thread owns a row), warps 8 and 11 issue
// products, warp 9 schedules and issues every copy (TMA, 128-byte swizzle, a ring of K and V tiles),
// warp 10 looks
// after hidden infinities.
//
// The row maximum is taken over with a slack of 2^8: O is rescaled only when the maximum has grown
// by more, since P and l hold such factors exactly as well and the quotient is the same.  P is
// rounded to bf16 (half a step, 2^-8 of a weight); l sums the unrounded weights in fp32.
//
// Hidden keys: scores are replaced by -inf.  An infinity or NaN in V would spread over 0 x inf, so a
// tile that some row does not see whole is cleaned of them first (noted by channel and key), and
// the rows that see them get them at the end.
#include <cfloat>

#include "kda_attn.cuh"
#include "kda_attn_tc.cuh"
#include "kda_attn_tile.cuh"
#include "kda_checks.cuh"
#include "kda_tc.cuh"

namespace kda {

using namespace attn;

namespace {

constexpr int kHalfRows = 128;
constexpr int kKeys = 128;
constexpr int kThreads = 384;
// warpgroups' registers after the split: 256 x 208 + 128 x 88 = 384 x 168, what the launch holds
constexpr int kRegsSoftmax = 208, kRegsOther = 88;

template <int D> struct Cfg {
    static constexpr int DP = D < 64 ? 64 : D;               // 32 channels are padded with zeros by the copies
    static constexpr int NB = DP / 64;                       // 64-channel blocks of a row
    static constexpr uint32_t BLK = 128 * 128;               // bytes of a block: 128 rows of 128 bytes
    static constexpr uint32_t TILE = NB * BLK;
    // P has columns of its own where there is room, and the next scores' product need not wait for it
    static constexpr bool APART = D < 128;
    // product warps: one for each half where the products are short, else one for both (see there)
    static constexpr int ISSUERS = D < 128 ? 2 : 1;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr uint32_t SMEM = 2 * TILE + STAGES * TILE + 1024;
};

struct Maps {
    CUtensorMap q, k, v;
};

struct TileInfo {
    int64_t start;
    int first, last, head, valid;
};

struct Shared {
    uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8], z_full[2], z_read[2], p_full[2], o_full[2], drained[2];
    uint64_t v_load[4], v_clean[4];  // V tiles with hidden keys, in turn: the ring holds at most four
    uint64_t info_full[2], info_empty[2], answer_full;
    alignas(16) uint64_t answer[2];
    TileInfo info[2], lost;  // lost: taken when a wait had given up, and not published
    uint32_t tmem, dead, dirty[2];
    uint32_t odd[2][3][128];  // by the tile's parity: first key with +inf, -inf, NaN in a channel
};

// What is noted in odd[]: the tile's turn (later turns are smaller, so that atomicMin prefers them)
// and the key's distance from the first key that is looked at.
__device__ __forceinline__ uint32_t odd_tag(uint32_t turn) { return 0x3fffffu - (turn & 0x3fffffu); }

// The grid index of a CTA that has not started yet, which then never starts: this CTA does its work
// (cluster launch control).  -1: none is left, and no further request is made.
__device__ __forceinline__ int take_tile(uint64_t* answer, uint64_t* bar, uint32_t asked)
{
    tc::fence_async_smem();  // the last answer was read
    tc::mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     tc::smem_u32(answer)),
                 "r"(tc::smem_u32(bar))
                 : "memory");
    if (!tc::mbar_wait(bar, asked & 1u, kTries)) return -1;
    const uint64_t lo = ((volatile uint64_t*)answer)[0], hi = ((volatile uint64_t*)answer)[1];
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tmov.b128 r, {%2, %3};\n\tmov.u32 %1, 0;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(got), "=&r"(x)
        : "l"(lo), "l"(hi));
    return got ? (int)x : -1;
}


}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kda_attn_prefill_tc_kernel(const AttnArgs a, const __grid_constant__ Maps maps, const int slots, const uint32_t tries)
{
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    unsigned char* sq = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* ring = sq + 2 * C::TILE;
    const int tid = threadIdx.x, lane = tid & 31;
    const int w = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
    const int tpt = kHalfRows / a.group;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.q_full[i], 1);
            tc::mbar_init(&sh.q_empty[i], 1);
            tc::mbar_init(&sh.z_full[i], 1);
            tc::mbar_init(&sh.z_read[i], 4);
            tc::mbar_init(&sh.p_full[i], 4);
            tc::mbar_init(&sh.o_full[i], 1);
            tc::mbar_init(&sh.drained[i], 1);
            tc::mbar_init(&sh.info_full[i], 1);
            tc::mbar_init(&sh.info_empty[i], 8 + C::ISSUERS + 1);  // softmax warps, products, cleaner
        }
        for (int i = 0; i < C::STAGES; ++i) {
            tc::mbar_init(&sh.kv_full[i], 1);
            tc::mbar_init(&sh.kv_empty[i], C::ISSUERS);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&sh.v_load[i], 1);
            tc::mbar_init(&sh.v_clean[i], 32);
        }
        tc::mbar_init(&sh.answer_full, 1);
        sh.dead = 0u;
        sh.info[0].valid = sh.info[1].valid = sh.lost.valid = 0;
        sh.dirty[0] = sh.dirty[1] = 0xffffffffu;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 2 * 3 * 128; i += kThreads) (&sh.odd[0][0][0])[i] = 0xffffffffu;
    if (w == 8) tc::tmem_alloc(&sh.tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sh.tmem;
    volatile uint32_t* dead = &sh.dead;

    // A role's next tile: waits until the scheduler has published it.  False: there is none (or a
    // wait gave up).  The role gives the slot back with done_tile.  (These waits alone, once a tile, take their
    // limit from the call: with a variable one in the inner waits long prompts took 3 % more.)
    struct Tile {
        int64_t start;
        int first, last, head, n0, n1, n, edge;
    };
    auto next_tile = [&](uint32_t turn, Tile& t) -> bool {
        if (!warp_wait(&sh.info_full[turn & 1], (turn >> 1) & 1u, tries)) {
            *dead = 1u;
            return false;
        }
        const TileInfo& i = sh.info[turn & 1];
        if (!i.valid || __any_sync(0xffffffffu, *dead != 0u)) return false;
        t.start = i.start;
        t.first = i.first;
        t.last = i.last;
        t.head = i.head;
        // key tiles of each half's tokens, and the first tile that is hidden in part from some row
        t.n0 = (min(t.first + tpt, t.last) + kKeys - 1) / kKeys;
        t.n1 = t.last > t.first + tpt ? (t.last + kKeys - 1) / kKeys : 0;
        t.n = max(t.n0, t.n1);
        t.edge = (t.first + 1) / kKeys;
        return true;
    };
    auto done_tile = [&](uint32_t turn) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.info_empty[turn & 1]);
    };

    if (w >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        Tile t;
        if (w == 9) {
            // ---- scheduler and copies.  This CTA's own tile, then tiles of CTAs that have not started yet: the
            // next is asked for once a tile's last copy has been issued, so that tiles go to whoever is nearly
            // free.  K0, Q, V0, K1, V1 ... through the ring, tile after tile.
            uint32_t it = 0, e = 0, qc[2] = {0, 0}, asked = 0;
            int idx = blockIdx.x;
            auto take = [&]() {
                int x = -1;
                if (lane == 0 && *dead == 0u) x = take_tile(sh.answer, &sh.answer_full, asked);
                ++asked;
                return __shfl_sync(0xffffffffu, x, 0);
            };
            for (uint32_t turn = 0;; ++turn, idx = take()) {
                TileInfo f{};
                for (;;) {
                    AttnTile x;
                    if (idx < 0) break;
                    // the longest rows of every sequence first
                    if (attn_tile(a, slots - 1 - idx / a.Hkv, 2 * tpt, x)) {
                        f = TileInfo{x.start, x.first, x.last, idx % a.Hkv, 1};
                        break;
                    }
                    idx = take();
                }
                if (!warp_wait(&sh.info_empty[turn & 1], ((turn >> 1) & 1u) ^ 1u, tries)) *dead = 1u;
                const bool over = __any_sync(0xffffffffu, *dead != 0u);  // the slot may hold a tile that is not finished
                if (lane == 0) {
                    (over ? sh.lost : sh.info[turn & 1]) = f;
                    tc::mbar_arrive(&sh.info_full[turn & 1]);
                }
                if (over || !f.valid) break;
                if (!next_tile(turn, t)) break;  // what the others see
                bool ok = true;
                if (lane == 0) {
                    for (int x = 0; x < 2 * t.n && ok; ++x, ++it) {
                        if (x == 1) {
                            for (int hf = 0; hf < 2 && ok; ++hf) {
                                if (hf == 1 && t.n1 == 0) break;
                                ok = tc::mbar_wait(&sh.q_empty[hf], (qc[hf] & 1u) ^ 1u, kTries) && *dead == 0u;
                                if (!ok) break;
                                ++qc[hf];
                                tc::mbar_arrive_expect_tx(&sh.q_full[hf], C::NB * (uint32_t)(tpt * a.group) * 128u);
                                for (int b = 0; b < C::NB; ++b)
                                    tc::tma_load_3d(sq + hf * C::TILE + b * C::BLK, &maps.q, 64 * b, t.head * a.group,
                                                    (int)(t.start + t.first + hf * tpt), &sh.q_full[hf]);
                            }
                            if (!ok) break;
                        }
                        const uint32_t st = it % C::STAGES;
                        ok = tc::mbar_wait(&sh.kv_empty[st], ((it / C::STAGES) & 1u) ^ 1u, kTries) && *dead == 0u;
                        if (!ok) break;
                        // a V tile that is cleaned reports to the cleaner alone; its own barrier only turns over
                        const bool clean = (x & 1) && (x >> 1) >= t.edge;
                        uint64_t* bar = clean ? &sh.v_load[e & 3] : &sh.kv_full[st];
                        if (clean) {
                            tc::mbar_arrive(&sh.kv_full[st]);
                            ++e;
                        }
                        tc::mbar_arrive_expect_tx(bar, C::TILE);
                        for (int b = 0; b < C::NB; ++b)
                            tc::tma_load_3d(ring + st * C::TILE + b * C::BLK, x & 1 ? &maps.v : &maps.k, 64 * b, t.head,
                                            (int)(t.start + (x >> 1) * kKeys), bar);
                    }
                }
                __syncwarp();
                if (!__all_sync(0xffffffffu, ok)) *dead = 1u;  // the next round publishes the end
            }
            // what was issued lands before the CTA ends, also where another role's wait gave up
            if (lane == 0) {
                for (int hf = 0; hf < 2; ++hf)
                    if (qc[hf] > 0) (void)tc::mbar_wait(&sh.q_full[hf], (qc[hf] - 1) & 1u, kTries);
                for (uint32_t i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
                    (void)tc::mbar_wait(&sh.kv_full[i % C::STAGES], (i / C::STAGES) & 1u, kTries);
                for (uint32_t i = e > 4 ? e - 4 : 0; i < e; ++i) (void)tc::mbar_wait(&sh.v_load[i & 3], (i >> 2) & 1u, kTries);
            }
        } else if (w == 8 || (w == 11 && C::ISSUERS == 2)) {
            // ---- products, in the order Z0(0) Z1(0) | O0(0) Z0(1) O1(0) Z1(1) | ... tile after tile; P apart:
            // Z(0) | Z(1) O(0) | Z(2) O(1) ... by a warp for each half.  (With 64 channels one warp's waits and
            // issues for both halves took longer than the products: 16384 tokens x 8 heads 261 us by one,
            // 236 by two; with 128 the fixed order is better: 2 x 8192, 16 of 4 heads 335 and 340.)
            constexpr int PER = 2 / C::ISSUERS;
            const int first_half = w == 8 ? 0 : 1;
            const uint32_t id_z = tc::idesc_bf16(128, kKeys), id_o = tc::idesc_bf16(128, C::DP) | (1u << 16);
            const uint32_t qa = tc::smem_u32(sq), ra = tc::smem_u32(ring);
            uint32_t base = 0, e = 0, qc[PER] = {}, pc[PER] = {}, rc[PER] = {};
            bool ok = true;
            auto full = [&](uint32_t it) { return warp_wait(&sh.kv_full[it % C::STAGES], (it / C::STAGES) & 1u); };
            auto issue_z = [&](int hf, uint32_t it) {
                const uint32_t k = ra + (it % C::STAGES) * C::TILE, q = qa + hf * C::TILE;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = (s >> 2) * C::BLK + (s & 3) * 32;
                    mma_ss(tm + 128 * hf, desc_qk(q + off), desc_qk(k + off), id_z, s > 0);
                }
                commit(&sh.z_full[hf]);
            };
            auto issue_o = [&](int hf, uint32_t it, bool first) {
                const uint32_t v = ra + (it % C::STAGES) * C::TILE;
#pragma unroll
                for (int s = 0; s < kKeys / 16; ++s)
                    mma_ts(tm + 256 + C::DP * hf, (C::APART ? tm + 384 + 64 * hf : tm + 128 * hf) + 8 * s, desc_v(v + s * 2048, D == 128 ? C::BLK : 1024u), id_o,
                           !first || s > 0);
            };
            // a slot is given back only after its copy was seen, also by a half that has no use for it
            auto release = [&](uint32_t it) { commit(&sh.kv_empty[it % C::STAGES]); };
            for (uint32_t turn = 0; ok && next_tile(turn, t); ++turn) {
                int nh[PER];
#pragma unroll
                for (int u = 0; u < PER; ++u) nh[u] = first_half + u ? t.n1 : t.n0;
                ok = full(base);
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int hf = first_half + u;
                    if (!ok || nh[u] == 0) continue;
                    ok = warp_wait(&sh.q_full[hf], qc[u]++ & 1u);
                    if (!ok) continue;
                    issue_z(hf, base);
                    if (nh[u] == 1) commit(&sh.q_empty[hf]);
                }
                if (ok) release(base);
                for (int j = 0; j < t.n && ok; ++j) {
                    const uint32_t iv = base + 2 * j + 1;
                    const bool more = j + 1 < t.n;
                    ok = !__any_sync(0xffffffffu, *dead != 0u) && (!more || full(iv + 1));
                    if constexpr (C::APART) {
                        // the next scores, as soon as the last ones have been read
#pragma unroll
                        for (int u = 0; u < PER; ++u) {
                            const int hf = first_half + u;
                            if (!ok || j >= nh[u]) continue;
                            ok = warp_wait(&sh.z_read[hf], rc[u]++ & 1u);
                            if (!ok || j + 1 >= nh[u]) continue;
                            tc::fence_after_sync();
                            issue_z(hf, iv + 1);
                            if (j + 2 == nh[u]) commit(&sh.q_empty[hf]);
                        }
                        if (ok && more) release(iv + 1);
                    }
                    ok = ok && full(iv);
                    if (j >= t.edge) {
                        if (ok && (j < nh[0] || j < nh[PER - 1])) ok = warp_wait(&sh.v_clean[e & 3], (e >> 2) & 1u);
                        ++e;
                    }
#pragma unroll
                    for (int u = 0; u < PER; ++u) {
                        const int hf = first_half + u;
                        if (!ok || j >= nh[u]) continue;
                        ok = warp_wait(&sh.p_full[hf], pc[u]++ & 1u);
                        if (!ok) continue;
                        tc::fence_after_sync();
                        issue_o(hf, iv, j == 0);
                        if (C::APART) {
                            commit(&sh.o_full[hf]);
                        } else if (j + 1 < nh[u]) {
                            issue_z(hf, iv + 1);  // its commit also covers O's product
                            if (j + 2 == nh[u]) commit(&sh.q_empty[hf]);
                        } else {
                            commit(&sh.o_full[hf]);
                        }
                    }
                    if (!ok) break;
                    release(iv);
                    if (!C::APART && more) release(iv + 1);
                }
                base += 2 * t.n;
                done_tile(turn);
            }
            if (!ok) *dead = 1u;
            commit(&sh.drained[first_half]);  // products in flight end before tensor memory is given back
            (void)warp_wait(&sh.drained[first_half], 0);
        } else if (w == 10) {
            // ---- V tiles with hidden keys: infinities and NaN leave the tile
            uint32_t base = 0, e = 0;
            for (uint32_t turn = 0; next_tile(turn, t); ++turn) {
                bool ok = true;
                for (int j = t.edge; j < t.n && ok; ++j, ++e) {
                    ok = warp_wait(&sh.v_load[e & 3], (e >> 2) & 1u) && !__any_sync(0xffffffffu, *dead != 0u);
                    if (!ok) break;
                    unsigned char* v = ring + (base + 2 * j + 1) % C::STAGES * C::TILE;
                    // eight vectors at a time: is there any exponent of all ones?  (Adding one to the
                    // exponent's last place then carries into the sign's.)
                    for (int i0 = lane; i0 < (int)C::TILE / 16; i0 += 8 * 32) {
                        uint4 u[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) u[q] = *reinterpret_cast<const uint4*>(v + (i0 + 32 * q) * 16);
                        uint32_t any = 0u;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            any |= (u[q].x & 0x7fff7fffu) + 0x00800080u;
                            any |= (u[q].y & 0x7fff7fffu) + 0x00800080u;
                            any |= (u[q].z & 0x7fff7fffu) + 0x00800080u;
                            any |= (u[q].w & 0x7fff7fffu) + 0x00800080u;
                        }
                        if ((any & 0x80008000u) == 0u) continue;
                        for (int q = 0; q < 8; ++q) {
                            const int i = i0 + 32 * q, row = (i >> 3) & 127, key = j * kKeys + row;
                            const int ch = (i >> 10) * 64 + (((i & 7) ^ (row & 7)) << 3);
                            uint16_t* x = reinterpret_cast<uint16_t*>(v + i * 16);
                            for (int c = 0; c < 8; ++c) {
                                const uint32_t b = x[c];
                                if ((b & 0x7f80u) != 0x7f80u) continue;
                                if (key < t.last) {
                                    sh.dirty[turn & 1] = odd_tag(turn);
                                    atomicMin(&sh.odd[turn & 1][b & 0x7fu ? 2 : b >> 15][ch + c],
                                              (odd_tag(turn) << 10) | (uint32_t)(key - t.edge * kKeys));
                                }
                                x[c] = 0;
                            }
                        }
                    }
                    tc::fence_async_smem();
                    tc::mbar_arrive(&sh.v_clean[e & 3]);
                }
                base += 2 * t.n;
                done_tile(turn);
                if (!ok) {
                    *dead = 1u;
                    break;
                }
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax: warpgroup hf owns half hf, a thread the row of its tensor-memory lane
        const int hf = w >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(w & 3) << 21;  // lane offset 32 (w % 4) in the address' upper half
        const uint32_t zt = tm + 128 * hf + lanes, ot = tm + 256 + C::DP * hf + lanes;
        const uint32_t pt = C::APART ? tm + 384 + 64 * hf + lanes : zt;
        const float cs = a.scale * 1.4426950408889634f;
        const int rt = r / a.group, rh = r - rt * a.group;
        const int wt = (32 * (w & 3)) / a.group;
        uint32_t zc = 0, oc = 0;
        Tile t;
        for (uint32_t turn = 0; next_tile(turn, t); ++turn) {
            const int nh = hf ? t.n1 : t.n0;
            const int first = t.first + hf * tpt;
            const int tok = first + rt;
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            bool gone = false;
            for (int j = 0; j < nh; ++j) {
                gone = !warp_wait(&sh.z_full[hf], zc++ & 1u);
                if (gone) break;
                tc::fence_after_sync();
                uint32_t z[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(zt + 32 * c, z + 32 * c);
                tc::tmem_wait_ld();
                if (C::APART) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sh.z_read[hf]);
                }
                if (j * kKeys + kKeys - 1 > first + wt) {
                    const int seen = tok + 1 - j * kKeys;
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i >= seen) z[i] = 0xff800000u;
                }
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(f_of(z[2 * e]), f_of(z[2 * e + 1]));
#pragma unroll
                for (int i = 8; i < 128; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], f_of(z[i + 2 * e]), f_of(z[i + 2 * e + 1]));
                const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * cs;
                float alpha = 1.f;
                if (j == 0) {
                    m = fmaxf(top, -FLT_MAX);  // scores that are all -inf weigh nothing, and keys that follow count
                } else if (top > m + 8.f) {
                    alpha = ex2(m - top);
                    m = top;
                }
                if (C::APART && j > 0) {  // the last P has been read, and O holds its product
                    gone = !warp_wait(&sh.o_full[hf], oc++ & 1u);
                    if (gone) break;
                    tc::fence_after_sync();
                }
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // (the products into O up to here have ended: with the scores that were waited for, or see above)
                    l2 = __fmul2_rn(l2, make_float2(alpha, alpha));
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(ot + 32 * c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(f_of(o[i]) * alpha);
                        tmem_st32(ot + 32 * c, o);
                    }
                }
                float mul = cs, off = -m;
                if (fabsf(m) > 1048576.f) {
                    // z cs - m rounds once; beyond 2^20 the rounding of m alone would show, and from 2^31 on pass the
                    // exponents that there are: round z cs as m was
#pragma unroll
                    for (int i = 0; i < 128; ++i) z[i] = __float_as_uint(__fmul_rn(f_of(z[i]), cs) - m);
                    mul = 1.f;
                    off = 0.f;
                }
                __syncwarp();
                const float2 cs2 = make_float2(mul, mul), nm2 = make_float2(off, off);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int e = 64 * q + 2 * i;
                        const float2 x = __ffma2_rn(make_float2(f_of(z[e]), f_of(z[e + 1])), cs2, nm2);
                        const float2 y = make_float2(ex2(x.x), ex2(x.y));
                        sum[i & 1] = __fadd2_rn(sum[i & 1], y);
                        p[i] = tc::pack_bf16(y.x, y.y);
                    }
                    tmem_st32(pt + 32 * q, p);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.p_full[hf]);
                l2 = __fadd2_rn(l2, __fadd2_rn(sum[0], sum[1]));
            }
            if (nh > 0) {
                if (!gone) gone = !warp_wait(&sh.o_full[hf], oc++ & 1u);
                gone = __any_sync(0xffffffffu, gone || *dead != 0u);
                if (gone) *dead = 1u;
                tc::fence_after_sync();
                const int rows = (min(first + tpt, t.last) - first) * a.group;
                const float inv = 1.f / (l2.x + l2.y);
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                     ((t.start + tok) * a.Hq + t.head * a.group + rh) * D;
                const bool dirty = *(volatile uint32_t*)&sh.dirty[turn & 1] == odd_tag(turn);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(ot + 32 * c, o);
                    tc::tmem_wait_ld();
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 x = __fmul2_rn(make_float2(f_of(o[2 * i]), f_of(o[2 * i + 1])), make_float2(inv, inv));
                        y[i] = tc::pack_bf16(x.x, x.y);
                    }
                    if (dirty) {
                        auto at = [&](int kind, int ch) {
                            const uint32_t e = sh.odd[turn & 1][kind][ch];
                            return (e >> 10) == odd_tag(turn) ? t.edge * kKeys + (int)(e & 1023u) : 0x7fffffff;
                        };
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int ch = 32 * c + 2 * i + e;
                                x[e] = attn_odd(f_of(o[2 * i + e]) * inv, tok, at(0, ch), at(1, ch), at(2, ch));
                            }
                            y[i] = tc::pack_bf16(x[0], x[1]);
                        }
                    }
                    if (r < rows) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4*>(out + 32 * c + 8 * i) = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                    }
                }
                tc::fence_before_sync();
            }
            done_tile(turn);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (w == 8) tc::tmem_dealloc(tm, 512);
    if (sh.dead != 0u) {
        // A wait gave up, which shows in the output: NaN in every row of the tiles that this CTA had taken and may
        // not have finished (the last two that were published, and one that was not).
        for (const TileInfo& x : {sh.info[0], sh.info[1], sh.lost}) {
            const int64_t row = (int64_t)a.group * D, n = x.valid ? (x.last - x.first) * row : 0;
            for (int64_t i = tid; i < n; i += kThreads)
                static_cast<__nv_bfloat16*>(a.out)[((x.start + x.first + i / row) * a.Hkv + x.head) * row + i % row] = __float2bfloat16_rn(NAN);
        }
    }
}

namespace {

bool encode_rows(CUtensorMap* m, const void* base, int d, int heads, int64_t tokens, int64_t stride, int box_heads,
                 int box_tokens)
{
    const TensorMapEncode enc = attn_tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t s)
{
    static_assert(Cfg<D>::SMEM + sizeof(Shared) <= 232448, "the tiles fit an SM");
    static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");
    const int tpt = kHalfRows / a.group;
    Maps maps;
    if (!encode_rows(&maps.q, a.q, D, a.Hq, a.T, a.qs, a.group, tpt) ||
        !encode_rows(&maps.k, a.k, D, a.Hkv, a.T, a.ks, 1, kKeys) ||
        !encode_rows(&maps.v, a.v, D, a.Hkv, a.T, a.vs, 1, kKeys))
        return cudaErrorInvalidValue;
    auto kern = kda_attn_prefill_tc_kernel<D>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, (int)Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t slots = attn_slots(a, 2 * tpt);
    kern<<<(unsigned)(slots * a.Hkv), kThreads, Cfg<D>::SMEM, s>>>(a, maps, (int)slots, checks::handoff_tries(kTries));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill_tc(const AttnArgs& a, cudaStream_t s)
{
    return a.d == 32 ? launch_d<32>(a, s) : a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace kda
