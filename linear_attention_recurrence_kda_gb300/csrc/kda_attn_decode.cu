// kda_attn_decode.cu -- the newest tokens of every sequence attend to the paged 8-bit cache
// (kda_attention_decode).
//
// A unit is one sequence, one key head and up to 8 NT rows (query heads of the group x tokens of the
// window); its keys come in tiles of 32.  The work is cut evenly: with W workers (warps) and all
// units' tiles in one line, each unit's after a gap for what its start costs, worker w takes the tiles at
// places [w total / W, (w + 1) total / W), whatever the lengths are.  A worker that holds all of a unit writes its output; otherwise it leaves (max, sum,
// unnormalised output) in the workspace, and the combine kernel joins the pieces in order.
//
// Per tile a warp does, with m16n8k16 f16 products and fp32 accumulators,
//   Z^T = scale ks (K Q^T),  m' = max(m, max z),  P = 2^(Z - m'),  O^T = O^T 2^(m - m') + V^T P^T,  l likewise
// Keys (and channels) are the products' 16 rows and queries their 8 columns: a group of 4 or 8 query
// heads then fills half as many products, registers and exponentials as with queries for rows.
// K and V codes become f16 exactly (e4m3 and int8 are subsets of f16).  A row of q is scaled by a
// power of two so that its largest value lies in [2^14, 2^15): bf16 values are then exact in f16 down
// to 2^-31 of the row's largest and end at 2^-38; fp32 values are split into two f16 parts (22 bits), as are their p.
// V's scale goes into O's unit: O is held in units of `vu`, which follows the pages' scales.  Of weights
// relative to the largest, what is cut off is at most half a step of f16 (2^-11 of the weight; fp32: 2^-22) or,
// far below the largest, 2^-32 (fp32: 2^-44) in units of `vu`, itself at most 64 times the page's own scale: over
// thousands of small weights, which together may count for as much as the largest, that stays small.
//
// HBM bounds it (2 d bytes per key and head, and a group of query heads per byte is far below the
// tensor cores' rate), so each warp keeps its own ring of tiles in flight by TMA with no barrier
// between warps; the 128-byte swizzle frees ldmatrix of bank conflicts.  What ldmatrix hands a thread
// sets the order of channels in a product: 16 bytes of a K row serve one k-step with q's channels
// permuted alike, and even and odd channels of V are rows 0-7 and 8-15 of a product.
#include <cuda_fp16.h>

#include "kda_attn.cuh"
#include "kda_attn_decode.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int kTile = 32;     // keys per tile
constexpr int kWarps = 4;     // workers per CTA
constexpr int kThreads = kWarps * 32;
// What a unit's start and end cost, in tiles.  Cut by tiles alone, the workers that hold short sequences end last.
// One token, 32 of 8 heads, us for a cost of 0, 2, 4, 8: 300 sequences of 20 to 900 keys 75, 61, 63, 65; 1000 of 10 to
// 300 102, 72, 75, 81; 256 of 512 to 576 60, 60, 60, 60.
constexpr int kUnitCost = 2;
constexpr uint32_t kCopyTries = 1u << 17;  // of up to 20 us each
constexpr float kLog2e = 1.4426950408889634f;

// By the unit's rows (8 nt): O takes NT d / 4 registers, so few rows leave room for three CTAs on an SM.
constexpr int ctas_of(int nt) { return nt == 1 ? 3 : 2; }
constexpr int stages_of(int nt, int d) { return (nt == 1 ? 2 : 3) * (d == 128 ? 1 : d == 64 ? 2 : 3); }

// Column tiles of 8 rows for a call's rows.  More than 16 rows make several units that read the same
// tiles, or another kernel takes them (kda_attn_window.cu).  Four column tiles, with O in 128 registers,
// took 202 us where two took 194 (28 rows, 64 sequences of 3150 keys, 8 heads).
inline int nt_of(int64_t rows) { return rows <= 8 ? 1 : 2; }

struct Maps {
    CUtensorMap k, v;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x)  // an 8 x 8 matrix of 16-bit values over the warp
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the part of (lo, hi) that their f16 rounding `h` leaves, times `up`
__device__ __forceinline__ uint32_t rest_f16(float lo, float hi, uint32_t h, float up = 1.f)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_f16((lo - f.x) * up, (hi - f.y) * up);
}

// What a weight's second part is multiplied by.  A weight p of at most 2^15 (2^7 for the largest when the
// reference was set) leaves a rest of at most 2^3, or 2^-25 where p is below f16's normal range; times 2^11 the
// rest keeps bits down to 2^-36.
constexpr float kRestUp = 2048.f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D>
__device__ __forceinline__ uint32_t swizzle(uint32_t off)
{
    return off ^ (((off >> 7) & (D == 128 ? 7u : D == 64 ? 3u : 1u)) << 4);
}

}  // namespace

template <typename TIO, int D, bool kE4m3, int NT>
__global__ void __launch_bounds__(kThreads, ctas_of(NT))
    kda_attn_decode_kernel(const AttnDecodeArgs a, const __grid_constant__ Maps maps, const int rows_max, const bool by_unit)
{
    constexpr bool kSplit = sizeof(TIO) == 4;  // fp32: q and p as two f16 parts
    constexpr int PARTS = kSplit ? 2 : 1;
    constexpr int kRows = 8 * NT;
    constexpr int NCH = D / 16;                // 16-byte chunks of a row = k-steps of K Q^T
    constexpr int S = stages_of(NT, D);
    constexpr uint32_t TB = kTile * D;         // bytes of a K (or V) tile
    extern __shared__ unsigned char smem_raw[];
    __shared__ int64_t prefix[kThreads + 1];  // places, and
    __shared__ int seqs[kThreads + 1];        // sequences that hold keys, before every run of sequences
    __shared__ alignas(8) uint64_t full[kWarps][S];
    __shared__ int pages[kWarps][S][2];
    __shared__ uint32_t flag;

    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, cq = lane & 3;
    unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* ring = smem + (size_t)w * S * 2 * TB;
    const DecodeLayout L = decode_layout(gridDim.x * kWarps, gridDim.x, rows_max, D);
    const int rows_all = a.L * a.group;
    const int row_tiles = (rows_all + kRows - 1) / kRows;
    const int64_t per_tile = (int64_t)a.Hkv * row_tiles;

    griddep_launch_dependents();
    if (tid == 0) flag = 0u;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) tc::mbar_init(&full[w][i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // The line that is cut evenly: each unit takes a place for every tile, after a gap for what its start and end
    // cost (where there are fewer units than workers, every piece has a start: no gap).
    const int gap = by_unit ? 0 : kUnitCost;
    auto places_of = [&](int tiles) { return tiles > 0 ? tiles + gap : 0; };
    const int chunk = (a.N + kThreads - 1) / kThreads;
    {
        int64_t sum = 0;
        int some = 0;
        bool bad = false;
        for (int i = 0; i < chunk; ++i) {
            const int n = tid * chunk + i;
            const int tiles = n < a.N ? tiles_of<kTile>(length_of(a, n, &bad)) : 0;
            sum += places_of(tiles);
            some += tiles > 0;
        }
        int64_t x = sum;
        int y = some;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t ux = __shfl_up_sync(0xffffffffu, x, off);
            const int uy = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) {
                x += ux;
                y += uy;
            }
        }
        prefix[tid + 1] = x;
        seqs[tid + 1] = y;
        if (tid == 0) {
            prefix[0] = 0;
            seqs[0] = 0;
        }
        __syncthreads();
        if (bad) atomicOr(&flag, kCheckBadSeqlens);
        int64_t before = 0;
        int some_before = 0;
        for (int i = 0; i < w; ++i) {
            before += prefix[(i + 1) * 32];
            some_before += seqs[(i + 1) * 32];
        }
        __syncthreads();
        prefix[tid + 1] = x + before;
        seqs[tid + 1] = y + some_before;
        __syncthreads();
    }
    // a sequence with nothing in the cache: rows of zeros
    const int64_t tokrow = (int64_t)a.Hq * D;
    for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
        if (length_of(a, n) == 0) {
            for (int i = tid; by_unit && i < per_tile; i += kThreads)
                reinterpret_cast<Record*>(a.ws + L.records)[n * per_tile + i].n = -1;
            TIO* o = static_cast<TIO*>(a.out) + (int64_t)n * a.L * tokrow;
            for (int64_t i = tid; i < a.L * tokrow; i += kThreads) st_io(o, i, 0.f);
        }
    }
    const int64_t total = prefix[kThreads] * per_tile;
    const int64_t W = min((int64_t)gridDim.x * kWarps, total);
    const int64_t worker = (int64_t)blockIdx.x * kWarps + w;
    Record* records = reinterpret_cast<Record*>(a.ws + L.records);
    float2* ml = reinterpret_cast<float2*>(a.ws + L.ml);
    float* po = reinterpret_cast<float*>(a.ws + L.o);
    Record mine{-1, 0, 0, 0, 0};
    Cursor cc;
    int64_t b1 = 0;
    int count = 0;
    if (worker < W) {
        const int64_t b0 = worker * total / W;
        b1 = (worker + 1) * total / W;
        // The first tile at or after a place, and the tiles before it: a run of sequences by bisection, then one
        // by one.  Lane 1 looks for the worker's end, the others for its start.
        const int64_t at_end = total - (int64_t)gap * seqs[kThreads] * per_tile;
        const int64_t b = lane == 1 && b1 < total ? b1 : b0;
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] * per_tile <= b) lo = mid;
            else hi = mid - 1;
        }
        int64_t at = prefix[lo] * per_tile;
        int64_t before = at - (int64_t)gap * seqs[lo] * per_tile;
        cc.n = lo * chunk;
        for (;;) {
            cc.len = length_of(a, cc.n);
            cc.tiles = tiles_of<kTile>(cc.len);
            const int64_t here = places_of(cc.tiles) * per_tile;
            if (at + here > b || cc.n + 1 >= a.N) break;
            at += here;
            before += cc.tiles * per_tile;
            ++cc.n;
        }
        const int64_t rest = b - at;
        const int64_t unit = rest / places_of(cc.tiles);
        cc.i = max(0, (int)(rest - unit * places_of(cc.tiles)) - gap);
        cc.h = (int)(unit / row_tiles);
        cc.rt = (int)(unit - (int64_t)cc.h * row_tiles);
        before += unit * cc.tiles + cc.i;
        const int64_t end = b1 < total ? __shfl_sync(0xffffffffu, before, 1) : at_end;
        count = (int)(end - __shfl_sync(0xffffffffu, before, 0));
        cc.n = __shfl_sync(0xffffffffu, cc.n, 0);
        cc.h = __shfl_sync(0xffffffffu, cc.h, 0);
        cc.rt = __shfl_sync(0xffffffffu, cc.rt, 0);
        cc.i = __shfl_sync(0xffffffffu, cc.i, 0);
        cc.tiles = __shfl_sync(0xffffffffu, cc.tiles, 0);
        cc.len = __shfl_sync(0xffffffffu, cc.len, 0);
    }
    if (count > 0) {
        Cursor ic = cc;
        const int box = min(kTile, a.c.page);  // rows of one copy
        const int page_shift = 31 - __clz(a.c.page);
        bool gone = false;                     // a wait gave up

        auto page_id = [&](const Cursor& c, int piece) -> int {
            const int key = c.i * kTile + piece * box;
            if (key >= c.len) return -1;
            const int p = __ldg(a.c.table + (int64_t)c.n * a.c.max_pages + (key >> page_shift));
            return p;
        };
        int p0 = page_id(ic, 0), p1 = box < kTile ? page_id(ic, 1) : -1;
        // the next tile of the issuing cursor into its stage
        auto issue = [&](int it) {
            const int st = it % S;
            bool ok0 = p0 >= 0 && p0 < a.c.num_pages, ok1 = p1 >= 0 && p1 < a.c.num_pages;
            const int key = ic.i * kTile;
            if ((key < ic.len && !ok0) || (box < kTile && key + box < ic.len && !ok1)) {
                if (lane == 0) atomicOr(&flag, kCheckBadSeqlens);
            }
            if (lane == 0) {
                // the scales' places; a page serves the whole tile, or 16 keys of it
                pages[w][st][0] = ok0 ? p0 * a.Hkv + ic.h : -1;
                pages[w][st][1] = box < kTile ? (ok1 ? p1 * a.Hkv + ic.h : -1) : pages[w][st][0];
                const uint32_t bytes = (uint32_t)((ok0 ? 1 : 0) + (ok1 ? 1 : 0)) * 2u * box * D;
                tc::mbar_arrive_expect_tx(&full[w][st], bytes);
                unsigned char* kd = ring + (size_t)st * 2 * TB;
                const int slot = key & (a.c.page - 1);
                if (ok0) {
                    tc::tma_load_3d(kd, &maps.k, 0, slot, p0 * a.Hkv + ic.h, &full[w][st]);
                    tc::tma_load_3d(kd + TB, &maps.v, 0, slot, p0 * a.Hkv + ic.h, &full[w][st]);
                }
                if (ok1) {
                    tc::tma_load_3d(kd + box * D, &maps.k, 0, 0, p1 * a.Hkv + ic.h, &full[w][st]);
                    tc::tma_load_3d(kd + TB + box * D, &maps.v, 0, 0, p1 * a.Hkv + ic.h, &full[w][st]);
                }
            }
            next_tile<kTile>(a, row_tiles, ic);
            if (it + 1 < count) {
                p0 = page_id(ic, 0);
                p1 = box < kTile ? page_id(ic, 1) : -1;
            }
        };
        int issued = 0;
        while (issued < count && issued < S) issue(issued++);

        // row 8 t + g of the unit as a product's second operand; this thread's results are of rows
        // 8 t + 2 cq + {0, 1}
        uint32_t qf[PARTS][NCH][NT][2];
        float O[NCH][NT][4];
        float m[NT][2], l[NT][2], f[NT][2], vu = 0.f, vtop = 0.f;
        int seen[NT][2];  // keys that the rows see
        bool begun = false;
        auto row_of = [&](int r, int& t, int& head) {
            const int R = cc.rt * kRows + r;
            t = R / a.group;
            head = cc.h * a.group + (R - t * a.group);
            return R < rows_all;
        };
        auto start_unit = [&]() {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                int t, head;
                const bool ok = row_of(8 * nt + g, t, head);
                const int sees = ok ? cc.len - a.L + t + 1 : 0;
                const TIO* q = static_cast<const TIO*>(a.q) + ((int64_t)cc.n * a.L + t) * a.qs + (int64_t)head * D + 4 * cq;
                float x[NCH][4], mx = 0.f;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    if constexpr (kSplit) {
                        const float4 v = ok ? *reinterpret_cast<const float4*>(q + 16 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
                        x[c][0] = v.x; x[c][1] = v.y; x[c][2] = v.z; x[c][3] = v.w;
                    } else {
                        const uint2 v = ok ? *reinterpret_cast<const uint2*>(q + 16 * c) : make_uint2(0u, 0u);
                        x[c][0] = __uint_as_float(v.x << 16);
                        x[c][1] = __uint_as_float(v.x & 0xffff0000u);
                        x[c][2] = __uint_as_float(v.y << 16);
                        x[c][3] = __uint_as_float(v.y & 0xffff0000u);
                    }
                }
#pragma unroll
                for (int c = 0; c < NCH; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[c][e]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // a power of two brings the row's largest value to [2^14, 2^15)
                int e = (int)((__float_as_uint(mx) >> 23) & 0xffu) - 127;
                e = min(max(e, -100), 127);
                const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);  // 2^(14 - e), exponents -113 .. 114
                const float fr = __uint_as_float((uint32_t)(127 + e - 14) << 23) * a.scale * kLog2e;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[c][i] *= up;
                    const uint32_t b0 = pack_f16(x[c][0], x[c][1]), b1 = pack_f16(x[c][2], x[c][3]);
                    qf[0][c][nt][0] = b0;
                    qf[0][c][nt][1] = b1;
                    if constexpr (kSplit) {
                        qf[PARTS - 1][c][nt][0] = rest_f16(x[c][0], x[c][1], b0);
                        qf[PARTS - 1][c][nt][1] = rest_f16(x[c][2], x[c][3], b1);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[c][nt][i] = 0.f;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    f[nt][u] = __shfl_sync(0xffffffffu, fr, 8 * cq + 4 * u);
                    seen[nt][u] = __shfl_sync(0xffffffffu, sees, 8 * cq + 4 * u);
                    m[nt][u] = -INFINITY;
                    l[nt][u] = 0.f;
                }
            }
            vu = vtop = 0.f;
        };
        // this segment's result: the output where the whole unit was here, else a piece
        auto finish = [&](bool whole, int slot) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float sum = l[nt][u];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    int t, head;
                    const int r = 8 * nt + 2 * cq + u;
                    if (!row_of(r, t, head)) continue;
                    const float mul = whole ? (sum == 0.f ? 0.f : vu / sum) : vu;
                    float* pd = po + ((int64_t)slot * rows_max + r) * D + 2 * g;
                    TIO* od = static_cast<TIO*>(a.out) + ((int64_t)cc.n * a.L + t) * tokrow + (int64_t)head * D + 2 * g;
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        const float2 o = make_float2(O[c][nt][u] * mul, O[c][nt][2 + u] * mul);  // channels 16 c + 2 g + {0, 1}
                        if (!whole) *reinterpret_cast<float2*>(pd + 16 * c) = o;
                        else if constexpr (kSplit) *reinterpret_cast<float2*>(od + 16 * c) = o;
                        else *reinterpret_cast<uint32_t*>(od + 16 * c) = tc::pack_bf16(o.x, o.y);
                    }
                    if (!whole && g == 0) ml[(int64_t)slot * rows_max + r] = make_float2(m[nt][u], sum);
                }
        };

        // a tile's scales are read while the tile before it is computed
        struct Scales {
            float k0, k1, v0, v1;
            bool has0, has1;
        };
        auto load_scales = [&](int st) {
            const int q0 = pages[w][st][0], q1 = pages[w][st][1];
            Scales x;
            x.has0 = q0 >= 0;
            x.has1 = q1 >= 0;
            x.k0 = x.has0 ? __ldg(a.c.k_scale + q0) : 0.f;
            x.v0 = x.has0 ? __ldg(a.c.v_scale + q0) : 0.f;
            x.k1 = x.has1 ? __ldg(a.c.k_scale + q1) : 0.f;
            x.v1 = x.has1 ? __ldg(a.c.v_scale + q1) : 0.f;
            return x;
        };
        __syncwarp();
        Scales next = load_scales(0);
        int it = 0;
        for (; it < count; ++it) {
            const int st = it % S;
            if (!begun) {
                start_unit();
                begun = true;
            }
            const float ks0 = next.k0, ks1 = next.k1, vs0 = next.v0, vs1 = next.v1;
            const bool has0 = next.has0, has1 = next.has1;
            if (it + 1 < count) next = load_scales((it + 1) % S);
            const bool arrived = tc::mbar_wait(&full[w][st], (uint32_t)(it / S) & 1u, kCopyTries);
            if (!__all_sync(0xffffffffu, arrived)) {
                gone = true;
                break;
            }
            unsigned char* kt = ring + (size_t)st * 2 * TB;
            unsigned char* vt = kt + TB;
            const uint32_t ka = tc::smem_u32(kt), va = tc::smem_u32(vt);
            const int key0 = cc.i * kTile;
            // rows of the tile that hold no key of this sequence: V must not reach the product
            const bool partial = key0 + kTile > cc.len || !has0 || !has1;
            if (partial) {
                for (int i = lane; i < (int)TB / 16; i += 32) {
                    const int r = i * 16 / D;
                    const bool dead = key0 + r >= cc.len || !(r < 16 ? has0 : has1);
                    // the swizzle permutes 16-byte chunks within a row (or within the rows that share 128 bytes)
                    if (dead) *reinterpret_cast<uint4*>(vt + swizzle<D>((uint32_t)i * 16)) = make_uint4(0u, 0u, 0u, 0u);
                }
                tc::fence_async_smem();
                __syncwarp();
            }
            // a key of the window is hidden from the window's earlier rows: a NaN in its value must
            // not reach them, so it leaves the tile here and joins the rows that see it below
            if (kE4m3 && a.L > 1 && key0 + kTile > cc.len - a.L + 1) {
                const int from = max(0, cc.len - a.L + 1 - key0), to = min(kTile, cc.len - key0);
                for (int r = from; r < to; ++r) {
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        // channels 16 c + 2 g + {0, 1}
                        const uint32_t u = *reinterpret_cast<const uint16_t*>(vt + swizzle<D>((uint32_t)(r * D + 16 * c)) + 2 * g);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (((u >> (8 * e)) & 0x7fu) != 0x7fu) continue;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    if (key0 + r < seen[nt][i]) O[c][nt][2 * e + i] = NAN;
                        }
                    }
                    __syncwarp();
                    for (int i = lane; i < D / 4; i += 32) {
                        uint32_t* at = reinterpret_cast<uint32_t*>(vt + swizzle<D>((uint32_t)(r * D + (i / 4) * 16)) + 4 * (i & 3));
                        *at &= ~__vcmpeq4(*at & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    }
                    __syncwarp();
                }
                tc::fence_async_smem();
            }

            // z of keys 16 k + g (values 0, 1) and 16 k + g + 8 (values 2, 3) for rows 2 cq + {0, 1}
            float z[2][NT][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[k][nt][i] = 0.f;
#pragma unroll
            for (int c = 0; c < NCH; c += 2) {
                uint32_t r[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) ldsm4(r[k], ka + swizzle<D>((uint32_t)((16 * k + (lane & 15)) * D + (c + (lane >> 4)) * 16)));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t kf[2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        widen<kE4m3>(r[k][2 * i], kf[k][0], kf[k][2]);
                        widen<kE4m3>(r[k][2 * i + 1], kf[k][1], kf[k][3]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        // fp32: the products' own sums are cut off, not rounded, so they add the parts of one
                        // step and ordinary additions the steps
                        float part[2][4] = {};
#pragma unroll
                        for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                mma_f16(kSplit ? part[k] : z[k][nt], kf[k], qf[p][c + i][nt][0], qf[p][c + i][nt][1]);
                        if constexpr (kSplit) {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int e = 0; e < 4; ++e) z[k][nt][e] += part[k][e];
                        }
                    }
                }
            }
            // Scores in base 2 (z s, rounded, so that however large they are the difference from the maximum is
            // at most zero), their maxima over the keys that are seen, and p = 2^(z s - m).  The reference m is set 2^7 below the largest score and moves
            // only when the maximum has grown by more than 2^8: p stays below 2^15, in f16's range and as
            // far up in it as can be, l and O hold the factor as well, and O is rarely rescaled.
            const bool edge = partial || key0 + kTile > cc.len - a.L + 1;
            // does a row that sees `n` keys see this thread's key 16 k + 8 e + g of the tile?
            auto sees = [&](int k, int e, int n) { return (k == 0 ? has0 : has1) && key0 + 16 * k + 8 * e + g < n; };
            float alpha[NT][2];
            bool moved = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float s0 = f[nt][u] * ks0, s1 = f[nt][u] * ks1;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        z[0][nt][2 * e + u] = __fmul_rn(z[0][nt][2 * e + u], s0);
                        z[1][nt][2 * e + u] = __fmul_rn(z[1][nt][2 * e + u], s1);
                    }
                    float top;
                    if (!edge) {
                        top = fmaxf(fmaxf(z[0][nt][u], z[0][nt][2 + u]), fmaxf(z[1][nt][u], z[1][nt][2 + u]));
                    } else {
                        top = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (sees(k, e, seen[nt][u])) top = fmaxf(top, z[k][nt][2 * e + u]);
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    const float now = top - m[nt][u] > 15.f ? top - 7.f : m[nt][u];
                    const float ref = now == -INFINITY ? 0.f : now;
                    alpha[nt][u] = ex2(m[nt][u] - ref);
                    moved |= now != m[nt][u];
                    m[nt][u] = now;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        z[0][nt][2 * e + u] = ex2(z[0][nt][2 * e + u] - ref);
                        z[1][nt][2 * e + u] = ex2(z[1][nt][2 * e + u] - ref);
                    }
                    if (edge) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!sees(k, e, seen[nt][u])) z[k][nt][2 * e + u] = 0.f;
                    }
                    l[nt][u] = l[nt][u] * alpha[nt][u] + ((z[0][nt][u] + z[0][nt][2 + u]) + (z[1][nt][u] + z[1][nt][2 + u]));
                }
            bool rescale = __any_sync(0xffffffffu, moved);
            // O^T += V^T P^T, sixteen keys (at most one page) at a time
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float vs = s == 0 ? vs0 : vs1;
                const float mag = fabsf(vs);
                // O's unit follows V's scale, from it to 64 times it, but never falls under 2^-40 of the
                // largest scale met (what is in O would grow past fp32): a page that far below
                // adds nothing that fp32 could hold
                float ratio = 1.f;
                if (!(mag <= vu && mag * 64.f >= vu) && mag > 0.f && mag < INFINITY) {
                    vtop = fmaxf(vtop, mag);
                    const float nu = fmaxf(mag, vtop * 9.094947e-13f);
                    ratio = vu == 0.f ? 0.f : vu / nu;
                    vu = nu;
                    rescale = true;
                }
                if (rescale) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float b0 = alpha[nt][0] * ratio, b1 = alpha[nt][1] * ratio;
                        alpha[nt][0] = alpha[nt][1] = 1.f;
#pragma unroll
                        for (int c = 0; c < NCH; ++c) {
                            O[c][nt][0] *= b0;
                            O[c][nt][1] *= b1;
                            O[c][nt][2] *= b0;
                            O[c][nt][3] *= b1;
                        }
                    }
                    rescale = false;
                }
                const float pv = vu == 0.f ? (vs == vs ? 0.f : vs) : vs / vu;
                uint32_t pf[PARTS][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float y0 = z[s][nt][2 * e] * pv, y1 = z[s][nt][2 * e + 1] * pv;
                        const uint32_t h = pack_f16(y0, y1);
                        pf[0][nt][e] = transpose8(h);
                        if constexpr (kSplit) pf[PARTS - 1][nt][e] = transpose8(rest_f16(y0, y1, h, kRestUp));
                    }
#pragma unroll
                for (int c = 0; c < NCH; c += 2) {
                    uint32_t r[4];
                    ldsm4t(r, va + swizzle<D>((uint32_t)((16 * s + (lane & 15)) * D + (c + (lane >> 4)) * 16)));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t vf[4];
                        widen<kE4m3>(__byte_perm(r[2 * i], r[2 * i + 1], 0x6420), vf[0], vf[2]);
                        widen<kE4m3>(__byte_perm(r[2 * i], r[2 * i + 1], 0x7531), vf[1], vf[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (kSplit) {
                                float part[2][4] = {};
#pragma unroll
                                for (int p = 0; p < PARTS; ++p) mma_f16(part[p], vf, pf[p][nt][0], pf[p][nt][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) O[c + i][nt][e] += fmaf(part[1][e], 1.f / kRestUp, part[0][e]);
                            } else {
                                mma_f16(O[c + i][nt], vf, pf[0][nt][0], pf[0][nt][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();  // the stage's tiles and pages[] have been read
            if (issued < count) issue(issued++);
            __syncwarp();  // lane 0's pages[] of that stage: with two stages the next iteration begins by reading them

            const bool unit_end = cc.i + 1 == cc.tiles;
            if (unit_end || it + 1 == count) {
                const bool here = (int64_t)cc.i <= it;  // the unit's first tile was this worker's
                const int64_t unit = (int64_t)cc.n * per_tile + (int64_t)cc.h * row_tiles + cc.rt;
                if (here && unit_end) {
                    finish(true, 0);
                    if (by_unit && lane == 0) records[unit].n = -1;
                } else {
                    finish(false, (int)(2 * worker + (here ? 1 : 0)));
                    if (here) {
                        const int64_t e = b1 - 1 + (cc.tiles - cc.i);  // past the unit's last place: this tile has b1 - 1
                        mine = Record{cc.n, cc.h, cc.rt, (int32_t)worker, (int32_t)((e * W + total - 1) / total - 1)};
                        if (by_unit && lane == 0) records[unit] = mine;
                    }
                }
                begun = false;
            }
            next_tile<kTile>(a, row_tiles, cc);
        }
        if (gone) {
            // units begun here that will not be finished: nothing to join
            for (bool begun_here = cc.i <= it; it < count; begun_here = cc.i == 0, ++it) {
                if (by_unit && begun_here && lane == 0)
                    records[(int64_t)cc.n * per_tile + (int64_t)cc.h * row_tiles + cc.rt].n = -1;
                next_tile<kTile>(a, row_tiles, cc);
            }
            // copies still in flight land in shared memory that the CTA gives back: wait for them
            for (int i = max(0, issued - S); i < issued; ++i) (void)tc::mbar_wait(&full[w][i % S], (uint32_t)(i / S) & 1u, kCopyTries);
            if (lane == 0) atomicOr(&flag, kCheckTimeout);
            mine.n = -1;
        }
    }
    if (!by_unit && lane == 0) records[worker] = mine;
    __syncthreads();
    if (tid == 0) reinterpret_cast<uint32_t*>(a.ws + L.flags)[blockIdx.x] = flag;
}

// Joins a unit's pieces: o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over the workers that hold
// one, in an order that the pieces' number fixes.  Block x looks after record x; `wpr` warps take a
// row's pieces in turn (many where few units were cut into many pieces), a lane D / 32 channels.
constexpr int kCombineWarps = 8;

template <typename TIO, int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    kda_attn_combine_kernel(const AttnDecodeArgs a, const int rows_max, const int workers, const int nflags, const int unit_rows,
                            const int wpr)
{
    constexpr int V = D / 32;
    __shared__ float part[kCombineWarps][D + 1];
    __shared__ uint32_t word;
    const DecodeLayout L = decode_layout(workers, nflags, rows_max, D);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        // the call's check word: every CTA's flags, so that nothing has to be cleared before the call
        if (threadIdx.x == 0) word = 0u;
        __syncthreads();
        uint32_t f = 0u;
        const uint32_t* flags = reinterpret_cast<const uint32_t*>(a.ws + L.flags);
        for (int i = threadIdx.x; i < nflags; i += blockDim.x) f |= flags[i];
        if (f) atomicOr(&word, f);
        __syncthreads();
        if (threadIdx.x == 0) *reinterpret_cast<uint32_t*>(a.ws) = word;
    }
    const Record rec = reinterpret_cast<const Record*>(a.ws + L.records)[blockIdx.x];
    if (rec.n < 0) return;
    const float2* ml = reinterpret_cast<const float2*>(a.ws + L.ml);
    const float* po = reinterpret_cast<const float*>(a.ws + L.o);
    const int pieces = rec.last - rec.first + 1;
    auto slot = [&](int i) { return (int64_t)(i == 0 ? 2 * rec.first + 1 : 2 * (rec.first + i)); };
    const int r = blockIdx.y * (blockDim.x / 32 / wpr) + w / wpr;
    const int R = rec.rt * unit_rows + r;
    const bool on = r < rows_max && R < a.L * a.group;
    float l = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
    if (on) {
        float m = -INFINITY;
        for (int i = lane; i < pieces; i += 32) m = fmaxf(m, ml[slot(i) * rows_max + r].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll 4
        for (int i = w % wpr; i < pieces; i += wpr) {
            const float2 x = ml[slot(i) * rows_max + r];
            const float* p = po + (slot(i) * rows_max + r) * D + lane * V;
            const float f = ex2(x.x - mu);
            l += x.y * f;
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
        if (w % wpr != 0) return;
        for (int i = 1; i < wpr; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] += part[w + i][lane * V + v];
            l += part[w + i][D];
        }
    }
    if (!on) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int t = R / a.group, head = rec.h * a.group + (R - t * a.group);
    TIO* od = static_cast<TIO*>(a.out) + (((int64_t)rec.n * a.L + t) * a.Hq + head) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) st_io(od, v, o[v] * inv);
}

namespace {

bool encode_codes(CUtensorMap* m, const void* base, const AttnDecodeArgs& a)
{
    const TensorMapEncode enc = attn_tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.c.page, (cuuint64_t)a.c.num_pages * a.Hkv};
    const cuuint64_t strides[2] = {(cuuint64_t)a.d, (cuuint64_t)a.d * a.c.page};
    const cuuint32_t box[3] = {(cuuint32_t)a.d, (cuuint32_t)(a.c.page < kTile ? a.c.page : kTile), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUtensorMapSwizzle sw = a.d == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : a.d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_32B;
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int decode_ctas(int nt) { return ctas_of(nt) * sm_count_of_current_device(); }

template <typename TIO, int D, bool kE4m3, int NT>
cudaError_t launch_nt(const AttnDecodeArgs& a, cudaStream_t s)
{
    Maps maps;
    if (!encode_codes(&maps.k, a.c.k, a) || !encode_codes(&maps.v, a.c.v, a)) return cudaErrorInvalidValue;
    constexpr int smem = kWarps * stages_of(NT, D) * 2 * kTile * D + 1024;
    static_assert(ctas_of(NT) * (smem + 3072) <= 233472, "the rings of an SM's CTAs fit");
    auto kern = kda_attn_decode_kernel<TIO, D, kE4m3, NT>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, smem);
    if (e != cudaSuccess) return e;
    const int64_t rows_all = (int64_t)a.L * a.group;
    const int rows = (int)(rows_all < 8 * NT ? rows_all : 8 * NT);
    const int64_t units = (int64_t)a.N * a.Hkv * ((rows_all + 8 * NT - 1) / (8 * NT));
    // no more workers than tiles that the page table can hold
    const double most = (double)units * (((int64_t)a.c.max_pages * a.c.page + kTile - 1) / kTile);
    const int full = decode_ctas(NT);
    const int ctas = most < (double)full * kWarps ? (int)((most + kWarps - 1) / kWarps) : full;
    const int workers = ctas * kWarps;
    const bool by_unit = units <= workers;
    kern<<<ctas, kThreads, smem, s>>>(a, maps, rows, by_unit);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_attn_join(a, sizeof(TIO) == 4 ? KDA_F32 : KDA_BF16, rows, 8 * NT, workers, ctas, by_unit, units, s);
}

template <typename TIO, int D, bool kE4m3>
cudaError_t launch_decode_d(const AttnDecodeArgs& a, cudaStream_t s)
{
    if (nt_of((int64_t)a.L * a.group) == 1) return launch_nt<TIO, D, kE4m3, 1>(a, s);
    return launch_nt<TIO, D, kE4m3, 2>(a, s);
}

template <typename TIO, bool kE4m3>
cudaError_t launch_decode_io(const AttnDecodeArgs& a, cudaStream_t s)
{
    if (a.d == 32) return launch_decode_d<TIO, 32, kE4m3>(a, s);
    if (a.d == 64) return launch_decode_d<TIO, 64, kE4m3>(a, s);
    return launch_decode_d<TIO, 128, kE4m3>(a, s);
}

}  // namespace

cudaError_t launch_attn_join(const AttnDecodeArgs& a, kda_dtype_t dt, int rows_max, int unit_rows, int workers, int flags,
                             bool by_unit, int64_t units, cudaStream_t s)
{
    // about workers / units pieces a unit: four or more a warp
    const int64_t pieces = by_unit ? workers / units : 1;
    const int wpr = pieces >= 32 ? 8 : pieces >= 16 ? 4 : pieces >= 8 ? 2 : 1;
    const int rpb = rows_max < kCombineWarps / wpr ? rows_max : kCombineWarps / wpr;
    const dim3 grid((unsigned)(by_unit ? units : workers), (unsigned)((rows_max + rpb - 1) / rpb));
    auto go = [&](auto kern) {
        return launch_dependent(kern, grid, dim3((unsigned)(rpb * wpr * 32)), 0, s, a, rows_max, workers, flags, unit_rows, wpr);
    };
    if (dt == KDA_F32)
        return a.d == 32 ? go(kda_attn_combine_kernel<float, 32>)
                         : a.d == 64 ? go(kda_attn_combine_kernel<float, 64>) : go(kda_attn_combine_kernel<float, 128>);
    return a.d == 32 ? go(kda_attn_combine_kernel<__nv_bfloat16, 32>)
                     : a.d == 64 ? go(kda_attn_combine_kernel<__nv_bfloat16, 64>) : go(kda_attn_combine_kernel<__nv_bfloat16, 128>);
}

size_t attn_decode_workspace_bytes(int64_t rows, int d, kda_dtype_t dt)
{
    const int nt = nt_of(rows);
    const size_t need = decode_layout(decode_ctas(nt) * kWarps, decode_ctas(nt), (int)(rows < 8 * nt ? rows : 8 * nt), d).total;
    const size_t window = attn_window_takes(rows, d, dt, INT64_MAX) ? attn_window_workspace_bytes(rows, d) : 0;
    return need > window ? need : window;  // which form runs depends on the cache
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, kda_dtype_t dt, cudaStream_t s)
{
    if (attn_window_takes((int64_t)a.L * a.group, a.d, dt, (int64_t)a.c.max_pages * a.c.page)) return launch_attn_window(a, s);
    const bool e4m3 = a.c.dtype == KDA_CACHE_E4M3;
    if (dt == KDA_BF16) return e4m3 ? launch_decode_io<__nv_bfloat16, true>(a, s) : launch_decode_io<__nv_bfloat16, false>(a, s);
    return e4m3 ? launch_decode_io<float, true>(a, s) : launch_decode_io<float, false>(a, s);
}

}  // namespace kda
