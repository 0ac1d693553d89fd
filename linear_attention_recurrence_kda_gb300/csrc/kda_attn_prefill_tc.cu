// kda_attn_prefill_tc.cu -- causal attention over packed prompts on the 5th-generation tensor cores:
// bf16, 64 or 128 channels (kda_attention_prefill).
//
//   Z = scale Q K^T,  P = 2^(Z log2 e - m),  O = sum P V,  o = O / l      per row, keys in tiles of 128
//
// A CTA holds two halves of 128 rows (the query heads of a group times 128 / group tokens each, so
// that a group shares every K and V tile) and walks the keys of both.  Products are tcgen05.mma with
// M = 128: Z from Q and K in shared memory, O += P V with P read from tensor memory and V taken
// token-major as it lies in shared memory.  Tensor memory: Z0 | Z1 | O0 | O1 (128 columns each at 128
// channels), P over the first half of its Z as packed bf16.
//
// The tensor cores are the bound: 4 x 128 x 128 x 128 multiply-adds per key tile and CTA, 2048 cycles
// at 4096 a cycle, against 1024 cycles of exponentials (32 a cycle) and about 800 of issue.  So the
// roles are split by warp and meet only at mbarriers: while one half's products run, the other
// half's softmax does.  Warps 0-3 and 4-7 own the halves (a thread owns a row), warp 8 issues every
// product, warp 9 every copy (TMA, 128-byte swizzle, a ring of K and V tiles), warps 10 and 11 look
// after hidden infinities.
//
// The row maximum is taken over with a slack of 2^8: O is rescaled only when the maximum has grown
// by more, since P and l hold such factors exactly as well and the quotient is the same.  P is
// rounded to bf16 (half a step, 2^-8 of a weight); l sums the unrounded weights in fp32.
//
// Hidden keys: scores are replaced by -inf.  An infinity or NaN in V would spread over 0 x inf, so a
// tile that some row does not see whole is cleaned of them first (noted by channel and key), and
// the rows that see them get them at the end.
#include "kda_attn.cuh"
#include "kda_attn_tile.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kHalfRows = 128;
constexpr int kKeys = 128;
constexpr int kThreads = 384;
constexpr uint32_t kTries = 1u << 17;  // of up to 20 us each
// warpgroups' registers after the split: 256 x 208 + 128 x 88 = 384 x 168, what the launch holds
constexpr int kRegsSoftmax = 208, kRegsOther = 88;

template <int D> struct Cfg {
    static constexpr int NB = D / 64;                        // 64-channel blocks of a row
    static constexpr uint32_t BLK = 128 * 128;               // bytes of a block: 128 rows of 128 bytes
    static constexpr uint32_t TILE = NB * BLK;
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr uint32_t SMEM = 2 * TILE + STAGES * TILE + 1024;
};

struct Maps {
    CUtensorMap q, k, v;
};

struct Shared {
    uint64_t q_full, kv_full[8], kv_empty[8], z_full[2], p_full[2], o_full[2], drained;
    uint64_t v_load[4], v_clean[4];  // V tile `edge` + e on barriers e % 4: the ring holds at most four
    uint32_t tmem, dead;
    int odd[3][128];
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// V as the second operand, token-major (its channels contiguous): 64-channel blocks BLK apart, groups
// of 8 tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr, uint32_t block)
{
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(block >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;  // SWIZZLE_128B
    return d;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float f_of(uint32_t u) { return __uint_as_float(u); }

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kda_attn_prefill_tc_kernel(const AttnArgs a, const __grid_constant__ Maps maps, const int slots)
{
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    unsigned char* sq = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* ring = sq + 2 * C::TILE;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int tpt = kHalfRows / a.group;

    // the longest rows of every sequence first
    const int h = blockIdx.x % a.Hkv;
    AttnTile t;
    if (!attn_tile(a, slots - 1 - (int)(blockIdx.x / a.Hkv), 2 * tpt, t)) return;
    // each half's tokens [first, last) and its number of key tiles
    const int last0 = min(t.first + tpt, t.last);
    const int n0 = (last0 + kKeys - 1) / kKeys;
    const int n1 = t.last > t.first + tpt ? (t.last + kKeys - 1) / kKeys : 0;
    const int n = max(n0, n1);
    const int edge = (t.first + 1) / kKeys;  // tiles from here on are hidden in part from some row

    if (tid == 0) {
        tc::mbar_init(&sh.q_full, 1);
        for (int i = 0; i < C::STAGES; ++i) {
            tc::mbar_init(&sh.kv_full[i], 1);
            tc::mbar_init(&sh.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.z_full[i], 1);
            tc::mbar_init(&sh.p_full[i], 128);
            tc::mbar_init(&sh.o_full[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&sh.v_load[i], 1);
            tc::mbar_init(&sh.v_clean[i], 64);
        }
        tc::mbar_init(&sh.drained, 1);
        sh.dead = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 3 * 128; i += kThreads) (&sh.odd[0][0])[i] = 0x7fffffff;
    if (w == 8) tc::tmem_alloc(&sh.tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sh.tmem;
    volatile uint32_t* dead = &sh.dead;

    if (w >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (w == 9 && lane == 0) {
            // ---- copies: Q, then K0 V0 K1 V1 ... through the ring
            tc::mbar_arrive_expect_tx(&sh.q_full, 2u * C::NB * (uint32_t)(tpt * a.group) * 128u);
            for (int hf = 0; hf < 2; ++hf)
                for (int b = 0; b < C::NB; ++b)
                    tc::tma_load_3d(sq + hf * C::TILE + b * C::BLK, &maps.q, 64 * b, h * a.group,
                                    (int)(t.start + t.first + hf * tpt), &sh.q_full);
            int it = 0;
            for (; it < 2 * n && *dead == 0u; ++it) {
                const int st = it % C::STAGES;
                if (!tc::mbar_wait(&sh.kv_empty[st], ((uint32_t)(it / C::STAGES) & 1u) ^ 1u, kTries)) {
                    *dead = 1u;
                    break;
                }
                // a V tile that is cleaned reports to the cleaners alone; its own barrier only turns over
                const int e = (it >> 1) - edge;
                const bool clean = (it & 1) && e >= 0;
                uint64_t* bar = clean ? &sh.v_load[e & 3] : &sh.kv_full[st];
                if (clean) tc::mbar_arrive(&sh.kv_full[st]);
                tc::mbar_arrive_expect_tx(bar, C::TILE);
                for (int b = 0; b < C::NB; ++b)
                    tc::tma_load_3d(ring + st * C::TILE + b * C::BLK, it & 1 ? &maps.v : &maps.k, 64 * b, h,
                                    (int)(t.start + (it >> 1) * kKeys), bar);
            }
            // after a wait that gave up, what was issued still lands before the CTA ends
            if (*dead) {
                (void)tc::mbar_wait(&sh.q_full, 0, kTries);
                for (int i = max(0, it - C::STAGES); i < it; ++i) {
                    (void)tc::mbar_wait(&sh.kv_full[i % C::STAGES], (uint32_t)(i / C::STAGES) & 1u, kTries);
                    const int e = (i >> 1) - edge;
                    if ((i & 1) && e >= 0) (void)tc::mbar_wait(&sh.v_load[e & 3], (uint32_t)(e >> 2) & 1u, kTries);
                }
            }
        } else if (w == 8 && lane == 0) {
            // ---- products, in the order Z0(0) Z1(0) | O0(0) Z0(1) O1(0) Z1(1) | ...
            const uint32_t id_z = tc::idesc_bf16(128, kKeys), id_o = tc::idesc_bf16(128, D) | (1u << 16);
            const uint32_t qa = tc::smem_u32(sq), ra = tc::smem_u32(ring);
            auto full = [&](int it) {
                const bool ok = tc::mbar_wait(&sh.kv_full[it % C::STAGES], (uint32_t)(it / C::STAGES) & 1u, kTries);
                if (!ok) *dead = 1u;
                return *dead == 0u;
            };
            auto issue_z = [&](int hf, int j) {
                const uint32_t k = ra + ((2 * j) % C::STAGES) * C::TILE, q = qa + hf * C::TILE;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = (s >> 2) * C::BLK + (s & 3) * 32;
                    tc::umma(tm + 128 * hf, tc::desc_sw128(q + off), tc::desc_sw128(k + off), id_z, s > 0);
                }
                tc::umma_commit(&sh.z_full[hf]);
            };
            auto issue_o = [&](int hf, int j) {
                const uint32_t v = ra + ((2 * j + 1) % C::STAGES) * C::TILE;
#pragma unroll
                for (int s = 0; s < kKeys / 16; ++s)
                    tc::umma_ts(tm + 256 + D * hf, tm + 128 * hf + 8 * s, desc_v(v + s * 2048, D == 128 ? C::BLK : 1024u),
                                id_o, j > 0 || s > 0);
                tc::umma_commit(&sh.o_full[hf]);
            };
            bool ok = tc::mbar_wait(&sh.q_full, 0, kTries) && full(0);
            if (!ok) *dead = 1u;
            if (ok) {
                issue_z(0, 0);
                if (n1 > 0) issue_z(1, 0);
                tc::umma_commit(&sh.kv_empty[0]);
            }
            for (int j = 0; j < n && ok; ++j) {
                ok = full(2 * j + 1);
                if (ok && j + 1 < n) ok = full(2 * j + 2);
                if (ok && j >= edge && !tc::mbar_wait(&sh.v_clean[(j - edge) & 3], (uint32_t)((j - edge) >> 2) & 1u, kTries)) ok = false;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int nh = hf ? n1 : n0;
                    if (!ok || j >= nh) continue;
                    if (!tc::mbar_wait(&sh.p_full[hf], (uint32_t)j & 1u, kTries) || *dead != 0u) {
                        ok = false;
                        continue;
                    }
                    tc::fence_after_sync();
                    issue_o(hf, j);
                    if (j + 1 < nh) issue_z(hf, j + 1);
                }
                if (!ok) break;
                tc::umma_commit(&sh.kv_empty[(2 * j + 1) % C::STAGES]);
                if (j + 1 < n) tc::umma_commit(&sh.kv_empty[(2 * j + 2) % C::STAGES]);
            }
            if (!ok) {
                *dead = 1u;
                tc::umma_commit(&sh.drained);  // products in flight end before tensor memory is given back
                (void)tc::mbar_wait(&sh.drained, 0, kTries);
            }
        } else if (w >= 10) {
            // ---- V tiles with hidden keys: infinities and NaN leave the tile
            const int me = tid - 320;
            for (int j = edge; j < n && *dead == 0u; ++j) {
                const int it = 2 * j + 1, st = it % C::STAGES;
                if (!tc::mbar_wait(&sh.v_load[(j - edge) & 3], (uint32_t)((j - edge) >> 2) & 1u, kTries)) {
                    *dead = 1u;
                    break;
                }
                unsigned char* v = ring + st * C::TILE;
#pragma unroll 8
                for (int i = me; i < (int)C::TILE / 16; i += 64) {
                    uint4* at = reinterpret_cast<uint4*>(v + i * 16);
                    const uint4 u = *at;
                    auto odd2 = [](uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; };
                    if (odd2(u.x) || odd2(u.y) || odd2(u.z) || odd2(u.w)) {
                        const int row = (i >> 3) & 127, key = j * kKeys + row;
                        const int ch = (i >> 10) * 64 + (((i & 7) ^ (row & 7)) << 3);
                        uint32_t x[4] = {u.x, u.y, u.z, u.w};
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t b = (x[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                            if ((b & 0x7f80u) != 0x7f80u) continue;
                            if (key < t.last) atomicMin(&sh.odd[b & 0x7fu ? 2 : b >> 15][ch + e], key);
                            x[e >> 1] &= ~(0xffffu << (16 * (e & 1)));
                        }
                        *at = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
                tc::fence_async_smem();
                tc::mbar_arrive(&sh.v_clean[(j - edge) & 3]);
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax: warpgroup hf owns half hf, a thread the row of its tensor-memory lane
        const int hf = w >> 2, r = tid & 127;
        const int nh = hf ? n1 : n0;
        const uint32_t lanes = (uint32_t)(w & 3) << 21;  // lane offset 32 (w % 4) in the address' upper half
        const uint32_t zt = tm + 128 * hf + lanes, ot = tm + 256 + D * hf + lanes;
        const int first = t.first + hf * tpt;
        const int tok = first + r / a.group;
        const int warp_first = first + (32 * (w & 3)) / a.group;
        const float cs = a.scale * 1.4426950408889634f;
        float m = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        bool gone = false;
        for (int j = 0; j < nh; ++j) {
            gone = !tc::mbar_wait(&sh.z_full[hf], (uint32_t)j & 1u, kTries) || *dead != 0u;
            if (__any_sync(0xffffffffu, gone)) break;
            tc::fence_after_sync();
            uint32_t z[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(zt + 32 * c, z + 32 * c);
            tc::tmem_wait_ld();
            if (j * kKeys + kKeys - 1 > warp_first) {
                const int seen = tok + 1 - j * kKeys;
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (i >= seen) z[i] = 0xff800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 128; i += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], fmaxf(f_of(z[i + 2 * e]), f_of(z[i + 2 * e + 1])));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs;
            float alpha = 1.f;
            if (j == 0) {
                m = top;
            } else if (top > m + 8.f) {
                alpha = ex2(m - top);
                m = top;
            }
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                l2 = __fmul2_rn(l2, make_float2(alpha, alpha));
                gone = !tc::mbar_wait(&sh.o_full[hf], (uint32_t)(j - 1) & 1u, kTries);
                if (__any_sync(0xffffffffu, gone)) break;
                tc::fence_after_sync();
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
            const float2 cs2 = make_float2(cs, cs), nm2 = make_float2(-m, -m);
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
                tmem_st32(zt + 32 * q, p);
            }
            l2 = __fadd2_rn(l2, __fadd2_rn(sum[0], sum[1]));
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(&sh.p_full[hf]);
        }
        if (nh > 0) {
            if (!__any_sync(0xffffffffu, gone))
                gone = !tc::mbar_wait(&sh.o_full[hf], (uint32_t)(nh - 1) & 1u, kTries) || *dead != 0u;
            gone = __any_sync(0xffffffffu, gone);
            if (gone) *dead = 1u;
            tc::fence_after_sync();
            const int rows = (min(first + tpt, t.last) - first) * a.group;
            const float inv = gone ? NAN : 1.f / (l2.x + l2.y);  // a wait that gave up shows in the output
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                 ((t.start + tok) * a.Hq + h * a.group + r % a.group) * D;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (!gone) {
                    tmem_ld32(ot + 32 * c, o);
                    tc::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                uint32_t y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int ch = 32 * c + 2 * i + e;
                        x[e] = attn_odd(f_of(o[2 * i + e]) * inv, tok, sh.odd[0][ch], sh.odd[1][ch], sh.odd[2][ch]);
                    }
                    y[i] = tc::pack_bf16(x[0], x[1]);
                }
                if (r < rows) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(out + 32 * c + 8 * i) = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (w == 8) tc::tmem_dealloc(tm, 512);
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t slots = attn_slots(a, 2 * tpt);
    kern<<<(unsigned)(slots * a.Hkv), kThreads, Cfg<D>::SMEM, s>>>(a, maps, (int)slots);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill_tc(const AttnArgs& a, cudaStream_t s)
{
    return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace kda
