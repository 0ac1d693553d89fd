// kda_attn_prefill.cu -- causal attention over packed prompts (kda_attention_prefill): the form for
// every size and type, on warp-level products.
//
//   z_ij = scale q_i . k_j,  p_ij = exp(z_ij - m_i),  o_i = sum_j p_ij v_j / sum_j p_ij,  j <= i
// with the maximum m_i and the sums carried along the keys in fp32 (one pass over K and V).
//
// A tile holds 128 rows: the query heads of one key head's group times 128 / group tokens, so that
// a group's heads share every K and V tile and the diagonal wastes little.  Eight warps take 16 rows
// each; keys come in tiles of 64.  bf16 operands enter m16n8k16 as they are; an fp32 operand x
// enters as x1 + x2 + x3 with x1 = bf16(x), x2 = bf16(x - x1), x3 = bf16(x - x1 - x2) (24 bits, fp32's
// range) and a product as its six terms down to 2^-16 of the first.
//
// Hidden keys: a score is replaced, not added to, and an infinity or NaN in V leaves the tile and is
// noted by channel and position; at the end it joins the rows that see it, so no row meets another
// sequence's or a later token's infinities.
#include "kda_attn.cuh"
#include "kda_attn_tile.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kRowsTile = 128;
constexpr int kKeys = 64;
constexpr int kThreads = 256;

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

// the bf16 parts of a pair; an infinity or NaN stays in the first alone
template <int PL>
__device__ __forceinline__ void split2(float lo, float hi, uint32_t (&part)[PL])
{
#pragma unroll
    for (int p = 0; p < PL; ++p) {
        const uint32_t h = tc::pack_bf16(lo, hi);
        part[p] = h;
        if (p + 1 < PL) {
            lo = fabsf(lo) < INFINITY ? lo - __uint_as_float(h << 16) : 0.f;
            hi = fabsf(hi) < INFINITY ? hi - __uint_as_float(h & 0xffff0000u) : 0.f;
        }
    }
}

// eight values of a row (zeros beyond it)
template <typename TIO>
__device__ __forceinline__ void load8(const TIO* p, bool ok, float (&x)[8])
{
    if constexpr (sizeof(TIO) == 2) {
        const uint4 u = ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = ok ? reinterpret_cast<const float4*>(p)[0] : z;
        const float4 b = ok ? reinterpret_cast<const float4*>(p)[1] : z;
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}

}  // namespace

template <typename TIO, int D>
__global__ void __launch_bounds__(kThreads, 1) kda_attn_prefill_kernel(const AttnArgs a, const int slots)
{
    constexpr int PL = sizeof(TIO) == 4 ? 3 : 1;
    constexpr int NK = D / 16;
    constexpr uint32_t QB = kRowsTile * D * 2, KB = kKeys * D * 2;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sq = smem_raw + ((128u - (tc::smem_u32(smem_raw) & 127u)) & 127u);
    unsigned char* sk = sq + PL * QB;
    unsigned char* sv = sk + PL * KB;
    __shared__ int odd[3][D];  // first key with +inf, -inf, NaN in the channel

    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
    const int tpt = kRowsTile / a.group;
    // the longest rows of every sequence first
    const int h = blockIdx.x % a.Hkv;
    AttnTile t;
    if (!attn_tile(a, slots - 1 - (int)(blockIdx.x / a.Hkv), tpt, t)) return;
    for (int i = tid; i < 3 * D; i += kThreads) (&odd[0][0])[i] = 0x7fffffff;

    // rows of q: row r is token t.first + r / group, query head h group + r % group
    const int rows = min(tpt, t.last - t.first) * a.group;
    constexpr int CH = D / 8;
    for (int i = tid; i < kRowsTile * CH; i += kThreads) {
        const int r = i / CH, c = i % CH;
        const int tok = r / a.group;
        float x[8];
        load8(static_cast<const TIO*>(a.q) + (t.start + t.first + tok) * a.qs + (int64_t)(h * a.group + r - tok * a.group) * D + c * 8,
              r < rows, x);
        uint32_t part[4][PL];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2<PL>(x[2 * e], x[2 * e + 1], part[e]);
#pragma unroll
        for (int p = 0; p < PL; ++p)
            *reinterpret_cast<uint4*>(sq + p * QB + tile_off<D>(r, c)) = make_uint4(part[0][p], part[1][p], part[2][p], part[3][p]);
    }

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

    for (int k0 = 0; k0 < t.last; k0 += kKeys) {
        __syncthreads();
        for (int i = tid; i < kKeys * CH; i += kThreads) {
            const int r = i / CH, c = i % CH;
            const bool ok = k0 + r < t.last;
            float x[8];
            uint32_t part[4][PL];
            load8(static_cast<const TIO*>(a.k) + (t.start + k0 + r) * a.ks + (int64_t)h * D + c * 8, ok, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) split2<PL>(x[2 * e], x[2 * e + 1], part[e]);
#pragma unroll
            for (int p = 0; p < PL; ++p)
                *reinterpret_cast<uint4*>(sk + p * KB + tile_off<D>(r, c)) = make_uint4(part[0][p], part[1][p], part[2][p], part[3][p]);
            load8(static_cast<const TIO*>(a.v) + (t.start + k0 + r) * a.vs + (int64_t)h * D + c * 8, ok, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!(fabsf(x[e]) < INFINITY)) {
                    atomicMin(&odd[x[e] != x[e] ? 2 : x[e] > 0.f ? 0 : 1][c * 8 + e], k0 + r);
                    x[e] = 0.f;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) split2<PL>(x[2 * e], x[2 * e + 1], part[e]);
#pragma unroll
            for (int p = 0; p < PL; ++p)
                *reinterpret_cast<uint4*>(sv + p * KB + tile_off<D>(r, c)) = make_uint4(part[0][p], part[1][p], part[2][p], part[3][p]);
        }
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
#pragma unroll
            for (int j = 0; j < kKeys / 16; ++j) {
#pragma unroll
                for (int p = 0; p < PL; ++p) {
                    uint32_t b[4];
                    ldsm4(b, ka + p * KB + tile_off<D>(16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1)));
#pragma unroll
                    for (int u = 0; u + p < PL; ++u) {
                        tc::mma16816(z[2 * j], qf[u], b[0], b[1]);
                        tc::mma16816(z[2 * j + 1], qf[u], b[2], b[3]);
                    }
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
        // m is the rounded maximum in base 2: every use takes the same value, so its rounding cancels
        const float n0 = fmaxf(m0, t0 * cs), n1 = fmaxf(m1, t1 * cs);
        const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
        const float a0 = ex2(m0 - u0), a1 = ex2(m1 - u1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j) {
            z[j][0] = ex2(fmaf(z[j][0], cs, -u0));
            z[j][1] = ex2(fmaf(z[j][1], cs, -u0));
            z[j][2] = ex2(fmaf(z[j][2], cs, -u1));
            z[j][3] = ex2(fmaf(z[j][3], cs, -u1));
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
            split2<PL>(z[2 * s][0], z[2 * s][1], x[0]);
            split2<PL>(z[2 * s][2], z[2 * s][3], x[1]);
            split2<PL>(z[2 * s + 1][0], z[2 * s + 1][1], x[2]);
            split2<PL>(z[2 * s + 1][2], z[2 * s + 1][3], x[3]);
            uint32_t pf[PL][4];
#pragma unroll
            for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) pf[p][i] = x[i][p];
#pragma unroll
            for (int c = 0; c < D / 8; c += 2) {
#pragma unroll
                for (int p = 0; p < PL; ++p) {
                    uint32_t b[4];
                    ldsm4t(b, va + p * KB + tile_off<D>(16 * s + (lane & 15), c + (lane >> 4)));
#pragma unroll
                    for (int u = 0; u + p < PL; ++u) {
                        tc::mma16816(O[c], pf[u], b[0], b[1]);
                        tc::mma16816(O[c + 1], pf[u], b[2], b[3]);
                    }
                }
            }
        }
    }
    __syncthreads();  // the notes in odd[] are complete
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = r0 + 8 * u;
        if (r >= rows) continue;
        const int tok = u ? tok1 : tok0;
        const float inv = 1.f / (u ? l1 : l0);
        TIO* o = static_cast<TIO*>(a.out) + ((t.start + tok) * a.Hq + h * a.group + r % a.group) * D + 2 * cq;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            float x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int ch = 8 * c + 2 * cq + e;
                x[e] = attn_odd(O[c][2 * u + e] * inv, tok, odd[0][ch], odd[1][ch], odd[2][ch]);
            }
            if constexpr (PL == 1) *reinterpret_cast<uint32_t*>(o + 8 * c) = tc::pack_bf16(x[0], x[1]);
            else *reinterpret_cast<float2*>(o + 8 * c) = make_float2(x[0], x[1]);
        }
    }
}

namespace {

template <typename TIO, int D>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t s)
{
    constexpr int PL = sizeof(TIO) == 4 ? 3 : 1;
    constexpr int smem = PL * (kRowsTile + 2 * kKeys) * D * 2 + 128;
    static_assert(smem + 4096 <= 232448, "the tiles fit an SM");
    auto kern = kda_attn_prefill_kernel<TIO, D>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, smem);
    if (e != cudaSuccess) return e;
    const int64_t slots = attn_slots(a, kRowsTile / a.group);
    kern<<<(unsigned)(slots * a.Hkv), kThreads, smem, s>>>(a, (int)slots);
    return cudaGetLastError();
}

template <typename TIO>
cudaError_t launch_io(const AttnArgs& a, cudaStream_t s)
{
    if (a.d == 32) return launch_d<TIO, 32>(a, s);
    if (a.d == 64) return launch_d<TIO, 64>(a, s);
    return launch_d<TIO, 128>(a, s);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs& a, kda_dtype_t dt, cudaStream_t s)
{
    if (dt == KDA_BF16 && a.d != 32) return launch_attn_prefill_tc(a, s);
    return dt == KDA_BF16 ? launch_io<__nv_bfloat16>(a, s) : launch_io<float>(a, s);
}

}  // namespace kda
