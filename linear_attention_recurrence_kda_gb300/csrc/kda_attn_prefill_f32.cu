// kda_attn_prefill_f32.cu -- causal attention over packed prompts in fp32 (kda_attention_prefill), on
// warp-level products.
//
//   z_ij = scale q_i . k_j,  p_ij = exp(z_ij - m_i),  o_i = sum_j p_ij v_j / sum_j p_ij,  j <= i
// with the maximum m_i and the sums carried along the keys in fp32 (one pass over K and V).
//
// A tile holds 64 rows (128 for groups of more than 64 heads): the query heads of one key head's group
// times 64 / group tokens, so that a group's heads share every K and V tile and the diagonal wastes
// little.  Warps take 16 rows each; keys come in tiles of half as many.  Two CTAs share an SM: with
// 128 rows and one CTA the longest rows of a few prompts set the time (prompts of 200 to 1300
// tokens, 10 of 2 heads of 128 channels, one CTA a tile: 208 us against 196).  With few tiles two CTAs of a cluster take
// a tile's key tiles in turn and join their sums through each other's shared memory (see launch_d).
// An fp32 operand x enters m16n8k16 bf16 products as x1 + x2 + x3 with
// x1 = bf16(x), finite wherever x is, x2 = bf16(x - x1), x3 = bf16(x - x1 - x2) (24 bits, fp32's range), a product as its six
// terms down to 2^-16 of the first.  Those products bound it: at 128 channels 12 a warp and key,
// about 8 cycles each on a sub-partition that two warps share; a tile's loads overlap with the products of
// the tile before it where the registers for them are there (up to 64 channels).
//
// Keys with an infinity or NaN take their scores from the fp32 values, one by one.
// Hidden keys: a score is replaced, not added to, and an infinity or NaN in V leaves the tile and is
// noted by channel and position; at the end it joins the rows that see it, so no row meets another
// sequence's or a later token's infinities.
#include "kda_attn.cuh"
#include "kda_attn_tile.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

template <int D>
__device__ __forceinline__ uint32_t tile_off(int row, int chunk)  // 16-byte chunk of a row of D 16-bit values
{
    const int x = D == 32 ? (row >> 1) & 3 : row & 7;
    return (uint32_t)(row * D * 2 + ((chunk ^ x) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int PL = 3;  // bf16 parts of a value

// The bf16 parts of a pair.  The first is at most the largest finite bf16 value: a value near fp32's largest
// would round to infinity, and its rest to the other one.
__device__ __forceinline__ void split2(float lo, float hi, uint32_t (&part)[PL])
{
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(part[0]) : "f"(hi), "f"(lo));
#pragma unroll
    for (int p = 0; p + 1 < PL; ++p) {
        lo -= __uint_as_float(part[p] << 16);
        hi -= __uint_as_float(part[p] & 0xffff0000u);
        part[p + 1] = tc::pack_bf16(lo, hi);
    }
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// eight values of a row (zeros beyond it)
struct Vec8 {
    float x[8];
    __device__ __forceinline__ void load(const float* p, bool ok)
    {
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = ok ? reinterpret_cast<const float4*>(p)[0] : z;
        const float4 b = ok ? reinterpret_cast<const float4*>(p)[1] : z;
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    // the three parts as three 16-byte chunks, `plane` bytes apart; true: there is an infinity or NaN among the values
    __device__ __forceinline__ bool store(unsigned char* at, uint32_t plane) const
    {
        uint32_t part[4][PL];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(x[2 * e], x[2 * e + 1], part[e]);
        float top = 0.f;  // 0 x finite is 0, 0 x anything else NaN
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaf(x[e], 0.f, top);
#pragma unroll
        for (int p = 0; p < PL; ++p)
            *reinterpret_cast<uint4*>(at + p * plane) = make_uint4(part[0][p], part[1][p], part[2][p], part[3][p]);
        return top != 0.f;
    }
};

// an address in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ uint32_t at_rank(const void* p, int rank)
{
    uint32_t y;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(tc::smem_u32(p)), "r"(rank));
    return y;
}

__device__ __forceinline__ uint32_t load_rank(uint32_t addr)
{
    uint32_t y;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(y) : "r"(addr) : "memory");
    return y;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace

template <int D, int ROWS, int KS>
__global__ void __launch_bounds__(2 * ROWS, 128 / ROWS) kda_attn_prefill_f32_kernel(const AttnArgs a, const int slots)
{
    constexpr int kRowsTile = ROWS, kKeys = ROWS / 2, kThreads = 2 * ROWS;
    constexpr int NK = D / 16;
    constexpr uint32_t QB = kRowsTile * D * 2, KB = kKeys * D * 2;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sq = smem_raw + ((128u - (tc::smem_u32(smem_raw) & 127u)) & 127u);
    unsigned char* sk = sq + PL * QB;
    unsigned char* sv = sk + PL * KB;
    __shared__ int odd[3][D];  // first key with +inf, -inf, NaN in the channel
    __shared__ uint32_t wild[2][kKeys / 32];  // by a key tile's turn: keys with an infinity or NaN in K

    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
    const int tpt = kRowsTile / a.group;
    // the longest rows of every sequence first
    const int rank = blockIdx.x % KS, place = blockIdx.x / KS;
    const int h = place % a.Hkv;
    AttnTile t;
    if (!attn_tile(a, slots - 1 - place / a.Hkv, tpt, t)) return;  // the whole cluster
    for (int i = tid; i < 3 * D; i += kThreads) (&odd[0][0])[i] = 0x7fffffff;
    if (tid < kKeys / 32) wild[0][tid] = 0u;

    // rows of q: row r is token t.first + r / group, query head h group + r % group
    const int rows = min(tpt, t.last - t.first) * a.group;
    constexpr int CH = D / 8;
    for (int i = tid; i < kRowsTile * CH; i += kThreads) {
        const int r = i / CH, c = i % CH;
        const int tok = r / a.group;
        Vec8 x;
        x.load(static_cast<const float*>(a.q) + (t.start + t.first + tok) * a.qs + (int64_t)(h * a.group + r - tok * a.group) * D + c * 8,
               r < rows);
        x.store(sq + tile_off<D>(r, c), QB);
    }
    // a key tile: NV vectors of K and of V a thread
    constexpr int NV = kKeys * CH / kThreads;
    constexpr bool kAhead = D <= 64;  // the registers hold the next tile while this one is computed
    Vec8 kx[NV], vx[NV];
    auto load = [&](int k0) {
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int i = tid + e * kThreads, r = i / CH, c = i % CH;
            const bool ok = k0 + r < t.last;
            kx[e].load(static_cast<const float*>(a.k) + (t.start + k0 + r) * a.ks + (int64_t)h * D + c * 8, ok);
            vx[e].load(static_cast<const float*>(a.v) + (t.start + k0 + r) * a.vs + (int64_t)h * D + c * 8, ok);
        }
    };
    constexpr int kStep = KS * kKeys;  // the cluster's CTAs take key tiles in turn
    if (kAhead) load(rank * kKeys);

    float O[D / 8][4];
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[c][i] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const float cs = a.scale * 1.4426950408889634f;
    const int r0 = 16 * w + g;
    const int tok0 = t.first + r0 / a.group, tok1 = t.first + (r0 + 8) / a.group;  // keys 0 .. tok are seen
    const int warp_last = t.first + (16 * w + 15) / a.group;
    const bool warp_on = 16 * w < rows;

    for (int k0 = rank * kKeys, turn = 0; k0 < t.last; k0 += kStep, turn ^= 1) {
        __syncthreads();
        if (tid < kKeys / 32) wild[turn ^ 1][tid] = 0u;  // the last tile's readers are past it
        if (!kAhead) load(k0);
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int i = tid + e * kThreads, r = i / CH, c = i % CH;
            if (kx[e].store(sk + tile_off<D>(r, c), KB)) atomicOr(&wild[turn][r / 32], 1u << (r % 32));
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                float& y = vx[e].x[x];
                if (!(fabsf(y) < INFINITY)) {
                    atomicMin(&odd[y != y ? 2 : y > 0.f ? 0 : 1][c * 8 + x], k0 + r);
                    y = 0.f;
                }
            }
            vx[e].store(sv + tile_off<D>(r, c), KB);
        }
        if (kAhead && k0 + kStep < t.last) load(k0 + kStep);
        __syncthreads();
        if (!warp_on || k0 > warp_last) continue;

        float z[kKeys / 8][4];
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[j][i] = 0.f;
        const uint32_t qa = tc::smem_u32(sq), ka = tc::smem_u32(sk), va = tc::smem_u32(sv);
#pragma unroll
        for (int s = 0; s < NK; ++s) {
            uint32_t qf[PL][4];
#pragma unroll
            for (int p = 0; p < PL; ++p) ldsm4(qf[p], qa + p * QB + tile_off<D>(16 * w + (lane & 15), 2 * s + (lane >> 4)));
            uint32_t b[PL][kKeys / 16][4];
#pragma unroll
            for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int j = 0; j < kKeys / 16; ++j)
                    ldsm4(b[p][j], ka + p * KB + tile_off<D>(16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1)));
            // The products' own sums are cut off, not rounded, so a step's terms are summed by them, the
            // small ones first, and the steps by ordinary additions (adding all to one accumulator
            // lost two bits: an error of 3.7e-6 where fp32 arithmetic has 8e-7).
            float part[kKeys / 8][4];
#pragma unroll
            for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[j][i] = 0.f;
#pragma unroll
            for (int order = PL - 1; order >= 0; --order)
#pragma unroll
                for (int p = 0; p <= order; ++p)
#pragma unroll
                    for (int j = 0; j < kKeys / 16; ++j) {
                        mma(part[2 * j], qf[order - p], b[p][j][0], b[p][j][1]);
                        mma(part[2 * j + 1], qf[order - p], b[p][j][2], b[p][j][3]);
                    }
#pragma unroll
            for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[j][i] += part[j][i];
        }
        // An infinity in a key would meet the parts of q one by one, which differ in sign or are zero: NaN, where q
        // itself gives one infinity.  Such keys' scores are formed from the fp32 values.
#pragma unroll 1
        for (int i = 0; i < kKeys / 32; ++i) {
#pragma unroll 1
            for (uint32_t m = wild[turn][i]; m != 0u; m &= m - 1u) {
                const int key = 32 * i + __ffs(m) - 1;
                const float* k = static_cast<const float*>(a.k) + (t.start + k0 + key) * a.ks + (int64_t)h * D;
                float s[2] = {0.f, 0.f};
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = min(r0 + 8 * u, rows - 1), tok = r / a.group;
                    const float* q = static_cast<const float*>(a.q) + (t.start + t.first + tok) * a.qs + (int64_t)(h * a.group + r - tok * a.group) * D;
#pragma unroll 1
                    for (int c = 0; c < D; c += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(q + c), y = *reinterpret_cast<const float4*>(k + c);
                        s[u] = fmaf(x.w, y.w, fmaf(x.z, y.z, fmaf(x.y, y.y, fmaf(x.x, y.x, s[u]))));
                    }
                }
#pragma unroll
                for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (8 * j + 2 * cq + e == key) {
                            z[j][e] = s[0];
                            z[j][2 + e] = s[1];
                        }
            }
        }
        if (k0 + kKeys - 1 > t.first + (16 * w) / a.group) {
#pragma unroll
            for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = k0 + 8 * j + 2 * cq + e;
                    if (key > tok0) z[j][e] = -INFINITY;
                    if (key > tok1) z[j][2 + e] = -INFINITY;
                }
        }
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
            t0 = fmaxf(t0, fmaxf(z[j][0], z[j][1]));
            t1 = fmaxf(t1, fmaxf(z[j][2], z[j][3]));
        }
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
        // m is the rounded maximum in base 2, and scores are rounded like it before it comes off: the largest weight is
        // one however large the scores are (unrounded they may differ from m by more than exponents hold)
        const float n0 = fmaxf(m0, t0 * cs), n1 = fmaxf(m1, t1 * cs);
        const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
        const float a0 = ex2(m0 - u0), a1 = ex2(m1 - u1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
            z[j][0] = ex2(__fmul_rn(z[j][0], cs) - u0);
            z[j][1] = ex2(__fmul_rn(z[j][1], cs) - u0);
            z[j][2] = ex2(__fmul_rn(z[j][2], cs) - u1);
            z[j][3] = ex2(__fmul_rn(z[j][3], cs) - u1);
            l0 += z[j][0] + z[j][1];
            l1 += z[j][2] + z[j][3];
        }
        if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                O[c][0] *= a0;
                O[c][1] *= a0;
                O[c][2] *= a1;
                O[c][3] *= a1;
            }
        }
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s) {
            uint32_t x[4][PL];
            split2(z[2 * s][0], z[2 * s][1], x[0]);
            split2(z[2 * s][2], z[2 * s][3], x[1]);
            split2(z[2 * s + 1][0], z[2 * s + 1][1], x[2]);
            split2(z[2 * s + 1][2], z[2 * s + 1][3], x[3]);
            uint32_t pf[PL][4];
#pragma unroll
            for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) pf[p][i] = x[i][p];
            constexpr int CG = 2;  // chunk pairs in turn
#pragma unroll
            for (int c = 0; c < D / 8; c += 2 * CG) {
                uint32_t b[PL][CG][4];
#pragma unroll
                for (int p = 0; p < PL; ++p)
#pragma unroll
                    for (int q = 0; q < CG; ++q) ldsm4t(b[p][q], va + p * KB + tile_off<D>(16 * s + (lane & 15), c + 2 * q + (lane >> 4)));
                float part[2 * CG][4];
#pragma unroll
                for (int q = 0; q < 2 * CG; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[q][i] = 0.f;
#pragma unroll
                for (int order = PL - 1; order >= 0; --order)
#pragma unroll
                    for (int p = 0; p <= order; ++p)
#pragma unroll
                        for (int q = 0; q < CG; ++q) {
                            mma(part[2 * q], pf[order - p], b[p][q][0], b[p][q][1]);
                            mma(part[2 * q + 1], pf[order - p], b[p][q][2], b[p][q][3]);
                        }
#pragma unroll
                for (int q = 0; q < 2 * CG; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[c + q][i] += part[q][i];
            }
        }
    }
    __syncthreads();  // the notes in odd[] are complete
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    int c0 = 0;                                       // this CTA writes chunks of 8 channels from here on
    const int(*odds)[D] = odd;
    if constexpr (KS > 1) {
        // The CTAs' sums, maxima and outputs lie in their shared memory, element-major; each CTA joins its share of the
        // channels, in the order of the ranks.
        __shared__ int odd_all[3][D];
        float* so = reinterpret_cast<float*>(sq);          // [D / 8][4][threads]
        float* st = so + D / 2 * kThreads;                 // m0, m1, l0, l1 [threads]
        static_assert((D / 2 + 4) * kThreads * 4 <= PL * 2 * (int)QB, "the sums fit where the tiles were");
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) so[(4 * c + i) * kThreads + tid] = O[c][i];
        st[tid] = m0;
        st[kThreads + tid] = m1;
        st[2 * kThreads + tid] = l0;
        st[3 * kThreads + tid] = l1;
        cluster_sync();
        float n0 = m0, n1 = m1, a0[KS], a1[KS];
#pragma unroll
        for (int x = 0; x < KS; ++x) {
            a0[x] = __uint_as_float(load_rank(at_rank(st + tid, x)));
            a1[x] = __uint_as_float(load_rank(at_rank(st + kThreads + tid, x)));
            n0 = fmaxf(n0, a0[x]);
            n1 = fmaxf(n1, a1[x]);
        }
        if (n0 == -INFINITY) n0 = 0.f;
        if (n1 == -INFINITY) n1 = 0.f;
        l0 = l1 = 0.f;
#pragma unroll
        for (int x = 0; x < KS; ++x) {
            a0[x] = ex2(a0[x] - n0);
            a1[x] = ex2(a1[x] - n1);
            l0 = fmaf(__uint_as_float(load_rank(at_rank(st + 2 * kThreads + tid, x))), a0[x], l0);
            l1 = fmaf(__uint_as_float(load_rank(at_rank(st + 3 * kThreads + tid, x))), a1[x], l1);
        }
        c0 = rank * (D / 8 / KS);
#pragma unroll
        for (int c = 0; c < D / 8 / KS; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < KS; ++x)
                    sum = fmaf(__uint_as_float(load_rank(at_rank(so + (4 * (c0 + c) + i) * kThreads + tid, x))), i < 2 ? a0[x] : a1[x], sum);
                O[c][i] = sum;
            }
        for (int i = tid; i < 3 * D; i += kThreads) {
            int first = 0x7fffffff;
#pragma unroll
            for (int x = 0; x < KS; ++x) first = min(first, (int)load_rank(at_rank(&odd[0][0] + i, x)));
            (&odd_all[0][0])[i] = first;
        }
        odds = odd_all;
        cluster_sync();  // nobody's shared memory is read any more, and odd_all is complete
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = r0 + 8 * u;
        if (r >= rows) continue;
        const int tok = u ? tok1 : tok0;
        const float inv = 1.f / (u ? l1 : l0);
        float* o = static_cast<float*>(a.out) + ((t.start + tok) * a.Hq + h * a.group + r % a.group) * D + 8 * c0 + 2 * cq;
#pragma unroll
        for (int c = 0; c < D / 8 / KS; ++c) {
            float x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int ch = 8 * (c0 + c) + 2 * cq + e;
                x[e] = attn_odd(O[c][2 * u + e] * inv, tok, odds[0][ch], odds[1][ch], odds[2][ch]);
            }
            *reinterpret_cast<float2*>(o + 8 * c) = make_float2(x[0], x[1]);
        }
    }
}

namespace {

template <int D, int ROWS, int KS>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s)
{
    constexpr int smem = PL * 2 * ROWS * D * 2 + 128;  // q, and K and V of half as many rows
    static_assert(128 / ROWS * (smem + 4096) <= 233472, "the tiles of an SM's CTAs fit");
    auto kern = kda_attn_prefill_f32_kernel<D, ROWS, KS>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, smem);
    if (e != cudaSuccess) return e;
    const int64_t slots = attn_slots(a, ROWS / a.group);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = KS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(slots * a.Hkv * KS));
    cfg.blockDim = dim3(2 * ROWS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, (int)slots);
}

// Up to three tiles an SM, two CTAs share a tile's keys: the longest tiles alone then set the time.  One and two
// CTAs a tile, 16 of 4 heads of 128 channels unless said, us: a prompt of 1200 tokens (304 tiles) 182 and 127; prompts
// of 200 to 1300, 10 of 2 heads (380 tiles) 181 and 158; one of 1800 (452 tiles) 279 and 286; of 2400 (604) 419 and
// 456; 8 of 1000 to 4000 4198 and 4551; 60 of 100, 10 of 2 heads (1120 tiles) 82 and 126.  (Four CTAs: 174 where two took
// 152.)  The lengths are not known here: a prompt of 1500 packed before those 60 begins last and takes 315 us by one
// and 266 by two, packed after them 231 and 262.
template <int D>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t s)
{
    if (a.group > 64) return launch_rows<D, 128, 1>(a, s);
    const bool split = attn_slots(a, 64 / a.group) * a.Hkv <= 3 * (int64_t)sm_count_of_current_device();
    return split ? launch_rows<D, 64, 2>(a, s) : launch_rows<D, 64, 1>(a, s);
}

}  // namespace

cudaError_t launch_attn_prefill_f32(const AttnArgs& a, cudaStream_t s)
{
    return a.d == 32 ? launch_d<32>(a, s) : a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace kda
