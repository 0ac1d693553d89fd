// kda_cache.cu -- keys and values of new tokens into a paged 8-bit cache (kda_cache_append).
//
// For a page and head with values x of the new tokens and MAX the code's range (448 or 127):
//   scale' = max(scale if the page already holds tokens, 2^e),  e >= -60 smallest with max|x| <= MAX 2^e
//   code   = rne(x / scale'),  older codes <- rne(code * scale / scale') where the scale grew
// A power of two makes x / scale exact and costs no precision in e4m3 (its steps are relative);
// when a scale grows, e4m3 codes only move by an exponent, so the second rounding touches
// subnormal codes alone.
//
// One CTA takes one page that the call writes, for one head and one of k and v.  The new rows are
// read once and wait in registers between the maximum and the rounding; the bytes bound it
// (io bytes read, one byte written per value).
#include <cuda_fp8.h>

#include "kda_attn.cuh"

namespace kda {

namespace {

constexpr int kVec = 8;        // values a thread holds of a row
constexpr int kMaxThreads = 256;
constexpr int kMaxIter = 8;    // 128 rows of 128 values over 256 threads of 8
constexpr int kMinExp = -60;

template <typename TIO> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&x)[kVec]) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Vec<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float (&x)[kVec]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

// two values to two codes (low byte first)
template <bool kE4m3>
__device__ __forceinline__ uint32_t encode2(float lo, float hi)
{
    if constexpr (kE4m3) {
        // saturating: infinities take +-448; NaN stays NaN
        return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
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
    uint2 r;
    r.x = encode2<kE4m3>(x[0] * mul, x[1] * mul) | (encode2<kE4m3>(x[2] * mul, x[3] * mul) << 16);
    r.y = encode2<kE4m3>(x[4] * mul, x[5] * mul) | (encode2<kE4m3>(x[6] * mul, x[7] * mul) << 16);
    return r;
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

template <typename TIO, bool kE4m3>
__global__ void __launch_bounds__(kMaxThreads) kda_cache_append_kernel(AppendArgs a, int slots_per_equal)
{
    __shared__ float warp_max[kMaxThreads / 32];
    const int h = blockIdx.y;
    const bool second = blockIdx.z != 0;
    const int page_tokens = a.c.page;
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
        const int64_t x = blockIdx.x;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)a.cu[mid] / page_tokens + 2LL * mid <= x) lo = mid;
            else hi = mid - 1;
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
    const TIO* src = static_cast<const TIO*>(second ? a.v : a.k) + (t0 + (p0 - first)) * (second ? a.vs : a.ks) +
                     (int64_t)h * a.d;
    const int64_t stride = second ? a.vs : a.ks;
    const int64_t ph = (int64_t)page * a.Hkv + h;
    uint8_t* codes = (second ? a.c.v : a.c.k) + ph * page_tokens * a.d;
    float* scale = (second ? a.c.v_scale : a.c.k_scale) + ph;

    const int vpr = a.d / kVec;  // threads per row
    const int r0 = threadIdx.x / vpr, c0 = (threadIdx.x % vpr) * kVec, rstep = blockDim.x / vpr;
    Vec<TIO> held[kMaxIter];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxIter; ++i) {
        const int r = r0 + i * rstep;
        if (r < rows) held[i].load(src + r * stride + c0);
    }
#pragma unroll
    for (int i = 0; i < kMaxIter; ++i) {
        if (r0 + i * rstep < rows) {
            float x[kVec];
            held[i].get(x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float m = fabsf(x[e]);
                amax = m < INFINITY ? fmaxf(amax, m) : amax;  // infinities and NaN set no scale
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    const float old = slot0 > 0 ? *scale : 0.f;  // read by every thread before one replaces it
    __syncthreads();
    for (int i = 0; i < (int)blockDim.x / 32; ++i) amax = fmaxf(amax, warp_max[i]);
    const float unit = fmaxf(scale_for<kE4m3>(amax), old);
    if (threadIdx.x == 0) *scale = unit;
    if (slot0 > 0 && unit != old) {  // the page's earlier rows move to the larger scale
        const float ratio = old / unit;
        for (int r = r0; r < slot0; r += rstep) {
            uint2* p = reinterpret_cast<uint2*>(codes + r * a.d + c0);
            const uint2 u = *p;
            float x[kVec];
            const uint32_t w[4] = {u.x & 0xffffu, u.x >> 16, u.y & 0xffffu, u.y >> 16};
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
#pragma unroll
    for (int i = 0; i < kMaxIter; ++i) {
        const int r = r0 + i * rstep;
        if (r < rows) {
            float x[kVec];
            held[i].get(x);
            *reinterpret_cast<uint2*>(codes + (slot0 + r) * a.d + c0) = encode8<kE4m3>(x, inv);
        }
    }
}

cudaError_t launch_cache_append(const AppendArgs& a, kda_dtype_t dt, cudaStream_t s)
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
    const dim3 grid((unsigned)slots, (unsigned)a.Hkv, 2);
    const bool e4m3 = a.c.dtype == KDA_CACHE_E4M3;
    if (dt == KDA_BF16) {
        if (e4m3) kda_cache_append_kernel<__nv_bfloat16, true><<<grid, threads, 0, s>>>(a, per_equal);
        else kda_cache_append_kernel<__nv_bfloat16, false><<<grid, threads, 0, s>>>(a, per_equal);
    } else {
        if (e4m3) kda_cache_append_kernel<float, true><<<grid, threads, 0, s>>>(a, per_equal);
        else kda_cache_append_kernel<float, false><<<grid, threads, 0, s>>>(a, per_equal);
    }
    return cudaGetLastError();
}

}  // namespace kda
