// kda_cache.cu -- keys and values of new tokens into a paged 8-bit cache (kda_cache_append), the keys as they are or turned
// by their positions (kda_rotary_append).
//
// For a page and head with values x of the new tokens and MAX the code's range (448 or 127):
//   scale' = max(scale if the page already holds tokens, 2^e),  e >= -60 smallest with max|x| <= MAX 2^e
//   code   = rne(x / scale'),  the page's other codes <- rne(code * scale / scale') where it grew
// A power of two makes x / scale exact and costs no precision in e4m3 (its steps are relative);
// when a scale grows, e4m3 codes only move by an exponent, so the second rounding touches
// subnormal codes alone.
//
// One CTA takes one page that the call writes and `heads` of its heads, k and v in turn.  The new rows
// are read once and wait in shared memory between the maximum and the rounding; the bytes bound it
// (io bytes read, one byte written per value).  Finding the page is a chain of four loads, about
// 2 us: a CTA that does one head and tensor spends most of its time there (69,632 tokens of 8 heads
// in bf16: 128 us, half the copy rate), so where there is work enough a CTA does several, the next
// ones' rows on their way by asynchronous copies while one is rounded (80 us, 5.3 TB/s, issue-bound; with the next
// one's rows in registers 114 us, for want of bytes in flight).
//
// Keys that turn: the sines and cosines of the page's tokens are formed once into a table in shared memory and serve the
// CTA's heads; a row's other channel of each pair lies with a neighbour in the same warp.  The turned values stay in
// registers, in fp32, between the maximum and the rounding.  Warps past the pages' CTAs turn q.  The same 69,632 tokens
// with 32 heads of q: 296 us for 231 us of bytes (5.3 TB/s), the pages alone 146; they are bound by issue and by their 96 KB
// a CTA, two to an SM.  Measured against (366 us when begun): the table read 8 bytes at a time, with its bank conflicts, 329;
// registers for three CTAs an SM, which spill, 330; q in a launch of its own 364.
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_attn.cuh"
#include "kda_rotary.cuh"

namespace kda {

namespace {

constexpr int kVec = 8;        // values a thread holds of a row
constexpr int kMaxThreads = 256;
constexpr int kMaxStages = 4;   // units whose rows are on their way or held
constexpr int kMinExp = -60;

// What a call does to its keys and queries on the way: nothing, or a turn.
struct AsTheyAre {
    static constexpr bool kTurns = false;
    static constexpr int kRows = 1;
};
template <int R> struct Turned {  // R: rows that a thread holds at most
    static constexpr bool kTurns = true;
    static constexpr int kRows = R;
    TurnArgs t;
    TurnRows q;
    int64_t tasks;  // warps of q
    int32_t groups, slots, table;  // CTAs along x that hold pages; bytes before the table of sines
};

// a thread's eight values of a row: asynchronous copy to shared memory, and back to registers
template <typename TIO>
__device__ __forceinline__ void fetch8(unsigned char* dst, const TIO* src)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll
    for (int i = 0; i < (int)sizeof(TIO) / 2; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 16 * i), "l"(reinterpret_cast<const char*>(src) + 16 * i) : "memory");
}

template <typename TIO>
__device__ __forceinline__ void get8(const unsigned char* p, float (&x)[kVec])
{
    if constexpr (sizeof(TIO) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}

// the largest magnitude among eight values and `top` (bf16: two halves side by side), as bits
template <typename TIO>
__device__ __forceinline__ uint32_t max8(const unsigned char* p, uint32_t top)
{
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    if constexpr (sizeof(TIO) == 2) {
        top = __vmaxu2(top, u.x & 0x7fff7fffu);
        top = __vmaxu2(top, u.y & 0x7fff7fffu);
        top = __vmaxu2(top, u.z & 0x7fff7fffu);
        return __vmaxu2(top, u.w & 0x7fff7fffu);
    } else {
        const uint4 v = reinterpret_cast<const uint4*>(p)[1];
        const uint32_t a = max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
        const uint32_t b = max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
        return max(top, max(a, b));
    }
}

template <typename TIO>
__device__ __forceinline__ float largest(uint32_t top)
{
    if constexpr (sizeof(TIO) == 2) return __uint_as_float(max(top << 16, top & 0xffff0000u));
    else return __uint_as_float(top);
}

// two values to two codes (low byte first)
template <bool kE4m3>
__device__ __forceinline__ uint32_t encode2(float lo, float hi)
{
    if constexpr (kE4m3) {
        // saturating: infinities take +-448; NaN stays NaN
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        const float a = lo == lo ? fminf(fmaxf(lo, -127.f), 127.f) : 0.f;
        const float b = hi == hi ? fminf(fmaxf(hi, -127.f), 127.f) : 0.f;
        return ((uint32_t)__float2int_rn(a) & 0xffu) | (((uint32_t)__float2int_rn(b) & 0xffu) << 8);
    }
}

template <bool kE4m3>
__device__ __forceinline__ float2 decode2(uint32_t c)
{
    if constexpr (kE4m3) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
        return __half22float2(*reinterpret_cast<const __half2*>(&h));
    } else {
        return make_float2((float)(int8_t)(c & 0xffu), (float)(int8_t)((c >> 8) & 0xffu));
    }
}

template <bool kE4m3>
__device__ __forceinline__ uint2 encode8(const float (&x)[kVec], float mul)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(mul, mul));
        c[i] = encode2<kE4m3>(y.x, y.y);
    }
    return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// The scale 2^e with the smallest e >= kMinExp that keeps amax within the code's range.  With
// amax = m 2^x and MAX = m' 2^y (both mantissas in [1/2, 1)) that is e = x - y + (m > m').
template <bool kE4m3>
__device__ __forceinline__ float scale_for(float amax)
{
    int x;
    const float m = frexpf(amax, &x);
    const int e = kE4m3 ? x - 9 + (m > 0.875f ? 1 : 0) : x - 7 + (m > 0.9921875f ? 1 : 0);
    return ldexpf(1.f, amax > 0.f ? max(e, kMinExp) : kMinExp);
}

}  // namespace

template <typename TIO, bool kE4m3, typename How>
__global__ void __launch_bounds__(kMaxThreads)
    kda_cache_append_kernel(AppendArgs a, int slots_per_equal, int heads, int stages, int stage_bytes, const __grid_constant__ How how)
{
    extern __shared__ __align__(16) unsigned char ring[];  // [stages][stage_bytes]
    __shared__ float warp_max[2][kMaxThreads / 32];
    const int page_tokens = a.c.page;
    if constexpr (How::kTurns) {
        if ((int)blockIdx.x >= how.slots) {
            const int64_t cta = (int64_t)((int)blockIdx.x - how.slots) * gridDim.y + blockIdx.y;
            const int64_t task = cta * (blockDim.x / 32) + (threadIdx.x >> 5);
            if (task < how.tasks) turn_task<TIO>(how.t, how.q, task, how.groups);
            return;
        }
    }
    // the sequence and which of its pages: sequence n owns the CTAs from cu[n] / page + 2 n on, at
    // least as many as pages it can touch (equal lengths: slots_per_equal each)
    int n, j;
    int64_t t0, count;
    if (a.cu == nullptr) {
        n = blockIdx.x / slots_per_equal;
        j = blockIdx.x - n * slots_per_equal;
        count = a.T / a.N;
        t0 = n * count;
    } else {
        int lo = 0, hi = a.N - 1;
        const int x = blockIdx.x;
        while (lo < hi) {  // 32 sequences a step
            const int step = (hi - lo + 31) / 32;
            const int at = lo + ((int)(threadIdx.x & 31) + 1) * step;
            const bool yes = at <= hi && (int64_t)a.cu[at] / page_tokens + 2LL * at <= x;
            lo += __popc(__ballot_sync(0xffffffffu, yes)) * step;
            hi = min(hi, lo + step - 1);
        }
        n = lo;
        t0 = a.cu[n];
        count = (int64_t)a.cu[n + 1] - t0;
        const int64_t jj = x - (t0 / page_tokens + 2LL * n);
        if (jj < 0 || count <= 0) return;
        j = (int)jj;
    }
    const int64_t len = a.lengths[n];
    const int64_t first = len - count;  // position of the first new token
    const bool bad = t0 < 0 || t0 + count > a.T || first < 0 || len > (int64_t)a.c.max_pages * page_tokens;
    const int64_t lp = first / page_tokens + j;  // the page's place in the sequence
    if (bad || lp * page_tokens >= len) {
        if (bad && a.check != nullptr && j == 0 && threadIdx.x == 0) atomicOr(a.check, kCheckBadSeqlens);
        return;
    }
    const int64_t p0 = max(lp * page_tokens, first), p1 = min((lp + 1) * page_tokens, len);
    const int slot0 = (int)(p0 - lp * page_tokens), rows = (int)(p1 - p0);
    const int page = a.c.table[(int64_t)n * a.c.max_pages + lp];
    if (page < 0 || page >= a.c.num_pages) {
        if (a.check != nullptr && threadIdx.x == 0) atomicOr(a.check, kCheckBadSeqlens);
        return;
    }
    const int h0 = blockIdx.y * heads;
    const int units = 2 * min(heads, a.Hkv - h0);  // k and v of every head
    const int vpr = a.d / kVec;                    // threads per row
    const int r0 = threadIdx.x / vpr, c0 = (threadIdx.x % vpr) * kVec, rstep = blockDim.x / vpr;
    // a thread fetches and reads the same places, so a unit's rows need no barrier
    const int mine_rows = r0 < rows ? (rows - r0 + rstep - 1) / rstep : 0;
    const int mine = (r0 * a.d + c0) * (int)sizeof(TIO), mine_step = rstep * a.d * (int)sizeof(TIO);
    auto load = [&](int u, int slot) {
        if (u < units) {
            const int64_t stride = u & 1 ? a.vs : a.ks;
            const TIO* src = static_cast<const TIO*>(u & 1 ? a.v : a.k) + (t0 + (p0 - first) + r0) * stride + (int64_t)(h0 + (u >> 1)) * a.d + c0;
            unsigned char* dst = ring + slot * stage_bytes + mine;
            for (int r = r0; r < rows; r += rstep, src += rstep * stride, dst += mine_step) fetch8(dst, src);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (How::kTurns) {
        // (cos, sin) of [rows][pairs], a thread's pairs two by two, so that neighbours read 16 bytes side by side
        float2* table = reinterpret_cast<float2*>(ring + how.table);
        const int pairs = how.t.rot >> 1, own = how.t.adjacent ? 2 : 3, parts = pairs >> own;  // 2^own pairs are a thread's
        for (int i = threadIdx.x; i < rows * pairs; i += blockDim.x) {
            const int r = i / pairs, pair = i - r * pairs;
            const int64_t token = t0 + (p0 - first) + r;
            const int position = how.t.positions != nullptr ? how.t.positions[(int64_t)how.t.axis[pair] * a.T + token] : (int)(p0 + r);
            float s, c;
            sincos_of(how.t, pair, position, s, c);
            table[r * pairs + 2 * (((pair & ((1 << own) - 1)) >> 1) * parts + (pair >> own)) + (pair & 1)] = make_float2(c, s);
        }
    }
    // A thread's eight channels of its row i, turned: the other channels of their pairs lie in the same row, eight
    // apart in the same warp.
    auto turned8 = [&](const unsigned char* held, int i, float (&x)[kVec]) {
        if constexpr (How::kTurns) {
            const unsigned char* at = held + i * mine_step;
            get8<TIO>(at, x);
            const int rot = how.t.rot, half = rot >> 1;
            if (c0 >= rot) return;
            const float4* row = reinterpret_cast<const float4*>(ring + how.table) + (r0 + i * rstep) * (half >> 1);
            if (how.t.adjacent) {
                row += c0 >> 3;
#pragma unroll
                for (int e = 0; e < kVec / 4; ++e) {
                    const float4 cs = row[e * (half >> 2)];
                    const float p = x[4 * e], q = x[4 * e + 2];
                    x[4 * e] = fmaf(p, cs.x, -x[4 * e + 1] * cs.y);
                    x[4 * e + 1] = fmaf(x[4 * e + 1], cs.x, p * cs.y);
                    x[4 * e + 2] = fmaf(q, cs.z, -x[4 * e + 3] * cs.w);
                    x[4 * e + 3] = fmaf(x[4 * e + 3], cs.z, q * cs.w);
                }
            } else {
                const bool up = c0 >= half;
                float y[kVec];
                get8<TIO>(at + (up ? -half : half) * (int)sizeof(TIO), y);
                row += (up ? c0 - half : c0) >> 3;
#pragma unroll
                for (int e = 0; e < kVec / 2; ++e) {
                    const float4 cs = row[e * (half >> 3)];
                    x[2 * e] = fmaf(x[2 * e], cs.x, y[2 * e] * (up ? cs.y : -cs.y));
                    x[2 * e + 1] = fmaf(x[2 * e + 1], cs.z, y[2 * e + 1] * (up ? cs.w : -cs.w));
                }
            }
        }
    };
    auto round = [&](int u, int slot) {
        const int64_t ph = (int64_t)page * a.Hkv + h0 + (u >> 1);
        uint8_t* codes = (u & 1 ? a.c.v : a.c.k) + ph * page_tokens * a.d;
        float* scale = (u & 1 ? a.c.v_scale : a.c.k_scale) + ph;
        const float old = slot0 > 0 ? *scale : 0.f;  // read by every thread before one replaces it
        const unsigned char* held = ring + slot * stage_bytes + mine;
        // magnitudes compare as integers; where the largest is an infinity or NaN, which set no scale,
        // the rows are looked through again for the largest that is neither
        uint32_t top = 0u;
        float turned[How::kRows][kVec];
        const bool turn = How::kTurns && (u & 1) == 0;
        float amax = 0.f;
        if (turn) {
            __syncwarp();  // the neighbours' copies have landed, too
#pragma unroll
            for (int i = 0; i < How::kRows; ++i) {
                if (i >= mine_rows) continue;
                turned8(held, i, turned[How::kTurns ? i : 0]);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    top = max(top, __float_as_uint(turned[How::kTurns ? i : 0][e]) & 0x7fffffffu);
                }
            }
            amax = __uint_as_float(top);
            if (!(amax < INFINITY)) {
                amax = 0.f;
#pragma unroll
                for (int i = 0; i < How::kRows; ++i) {
                    if (i >= mine_rows) continue;
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const float m = fabsf(turned[How::kTurns ? i : 0][e]);
                        amax = m < INFINITY ? fmaxf(amax, m) : amax;
                    }
                }
            }
        } else {
#pragma unroll 4
            for (int i = 0; i < mine_rows; ++i) top = max8<TIO>(held + i * mine_step, top);
            amax = largest<TIO>(top);
        }
        if (!turn && !(amax < INFINITY)) {
            amax = 0.f;
            for (int i = 0; i < mine_rows; ++i) {
                float x[kVec];
                get8<TIO>(held + i * mine_step, x);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float m = fabsf(x[e]);
                    amax = m < INFINITY ? fmaxf(amax, m) : amax;
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        if ((threadIdx.x & 31) == 0) warp_max[u & 1][threadIdx.x >> 5] = amax;
        __syncthreads();  // (the other buffer's readers are past it: one barrier a unit)
        for (int i = 0; i < (int)blockDim.x / 32; ++i) amax = fmaxf(amax, warp_max[u & 1][i]);
        const float unit = fmaxf(scale_for<kE4m3>(amax), old);
        if (threadIdx.x == 0) *scale = unit;
        if (slot0 > 0 && unit != old) {  // the page's other rows move to the larger scale
            const float ratio = old / unit;
            for (int r = r0; r < page_tokens; r += rstep) {
                if (r >= slot0 && r < slot0 + rows) continue;
                uint2* p = reinterpret_cast<uint2*>(codes + r * a.d + c0);
                const uint2 q = *p;
                float x[kVec];
                const uint32_t w[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = decode2<kE4m3>(w[e]);
                    x[2 * e] = f.x;
                    x[2 * e + 1] = f.y;
                }
                *p = encode8<kE4m3>(x, ratio);
            }
        }
        const float inv = 1.f / unit;
        uint8_t* dst = codes + (slot0 + r0) * a.d + c0;
        if (turn) {
#pragma unroll
            for (int i = 0; i < How::kRows; ++i)
                if (i < mine_rows) *reinterpret_cast<uint2*>(dst + i * rstep * a.d) = encode8<kE4m3>(turned[How::kTurns ? i : 0], inv);
            return;
        }
#pragma unroll 4
        for (int i = 0; i < mine_rows; ++i) {
            float x[kVec];
            get8<TIO>(held + i * mine_step, x);
            *reinterpret_cast<uint2*>(dst + i * rstep * a.d) = encode8<kE4m3>(x, inv);
        }
    };
    for (int u = 0; u < stages - 1; ++u) load(u, u);
    if constexpr (How::kTurns) __syncthreads();  // the table
    int slot = 0, ahead = stages - 1;
    for (int u = 0; u < units; ++u) {
        load(u + stages - 1, ahead);
        ahead = ahead + 1 == stages ? 0 : ahead + 1;
        switch (stages) {  // all but the copies of the units after this one
            case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
            case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
            default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        }
        round(u, slot);
        slot = slot + 1 == stages ? 0 : slot + 1;
    }
}

namespace {

template <typename How>
cudaError_t launch(const AppendArgs& a, How how, kda_dtype_t dt, cudaStream_t s)
{
    // a call of at most c tokens a sequence holds min(c, page) rows in a CTA, so that few tokens
    // take few threads (one token of 128 channels: one warp)
    const int64_t c = a.cu == nullptr ? a.T / a.N : a.T;
    const int per_equal = c == 1 ? 1 : (int)(c / a.c.page + 2);
    const int64_t slots = a.cu == nullptr ? (int64_t)a.N * per_equal : a.T / a.c.page + 2LL * a.N;
    if (slots > 2147483647LL) return cudaErrorInvalidValue;
    const int64_t rows = c < a.c.page ? c : a.c.page;
    int threads = (int)((rows * (a.d / kVec) + 31) / 32 * 32);
    if (threads > kMaxThreads) threads = kMaxThreads;
    const int stage_bytes = (int)rows * a.d * (dt == KDA_BF16 ? 2 : 4);  // at most 64 KB
    int stages = 65536 / stage_bytes;
    stages = stages > kMaxStages ? kMaxStages : stages < 2 ? 2 : stages;
    int smem = stages * stage_bytes, resident = 8;
    if constexpr (How::kTurns) {
        how.slots = (int)slots;
        how.table = smem;
        smem += (int)rows * how.t.rot / 2 * (int)sizeof(float2);  // at most 64 KB
        resident = std::min(resident, 229376 / smem);
    }
    // Several heads a CTA while about eight CTAs an SM remain, or as many as it holds: where the table leaves room for two,
    // more CTAs only read, look up and form again what one does for all heads (256 single tokens of 8 and 32 heads:
    // 31.5 us with the eight, 21 with the two; 69,632 tokens: 366 and 329).
    int heads = 1;
    while (2 * heads <= a.Hkv && slots * ((a.Hkv + 2 * heads - 1) / (2 * heads)) >= (int64_t)resident * sm_count_of_current_device()) heads *= 2;
    dim3 grid((unsigned)slots, (unsigned)((a.Hkv + heads - 1) / heads));
    if constexpr (How::kTurns) {
        if (how.q.heads[0] > 0) how.tasks = turn_tasks(how.t, how.q, &how.groups);
        const int64_t per = (int64_t)grid.y * (threads / 32);  // of q's warps that a place of x holds
        const int64_t x = slots + (how.tasks + per - 1) / per;
        if (x > 2147483647LL) return cudaErrorInvalidValue;
        grid.x = (unsigned)x;
    }
    auto go = [&](auto kern, SmemLimit& limit) {
        const cudaError_t e = limit.raise(kern, (How::kTurns ? 3 : 2) * 65536);
        if (e == cudaSuccess) kern<<<grid, threads, smem, s>>>(a, per_equal, heads, stages, stage_bytes, how);
        return e;
    };
    static SmemLimit limit[4];
    const bool e4m3 = a.c.dtype == KDA_CACHE_E4M3;
    const cudaError_t e = dt == KDA_BF16 ? (e4m3 ? go(kda_cache_append_kernel<__nv_bfloat16, true, How>, limit[0])
                                                 : go(kda_cache_append_kernel<__nv_bfloat16, false, How>, limit[1]))
                                         : (e4m3 ? go(kda_cache_append_kernel<float, true, How>, limit[2])
                                                 : go(kda_cache_append_kernel<float, false, How>, limit[3]));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, kda_dtype_t dt, cudaStream_t s) { return launch(a, AsTheyAre{}, dt, s); }

cudaError_t launch_rotary_append(const AppendArgs& a, const TurnArgs& t, const TurnRows& q, kda_dtype_t dt, cudaStream_t s)
{
    auto go = [&](auto how) {
        how.t = t;
        how.q = q;
        return launch(a, how, dt, s);
    };
    // (four rows a thread where they do: 294 us for the 69,632 tokens, 305 with eight's registers)
    return a.c.page * (a.d / kVec) <= 4 * kMaxThreads ? go(Turned<4>{}) : go(Turned<8>{});
}

}  // namespace kda
