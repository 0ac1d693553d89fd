// kda_attn_extend.cu -- chunks of new tokens, of any length each, attend to the paged 8-bit cache
// (kda_attention_extend).
//
//   z_j = scale (q . k_j),   o = sum_j e^(z_j) v_j / sum_j e^(z_j)       over the keys j <= place of the row's token
//
// A warp takes a row: its keys one by one, running maximum and sum, the channels spread over the lanes.
#include <type_traits>

#include <cuda_fp16.h>

#include "kda_attn.cuh"
#include "kda_attn_decode.cuh"

namespace kda {

namespace {
constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
}

template <typename TIO, int D, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) kda_attn_extend_kernel(const AttnExtendArgs a)
{
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t token = row / a.Hq;
    const int head = (int)(row - token * a.Hq), h = head / a.group;
    if (token >= a.T) return;
    int64_t start, end;
    int n;
    if (a.cu == nullptr) {
        const int64_t len = a.T / a.N;
        n = (int)(token / len);
        start = n * len;
        end = start + len;
    } else {
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
            lo += __popc(__ballot_sync(0xffffffffu, at <= hi && a.cu[at] <= token)) * step;
            hi = min(hi, lo + step - 1);
        }
        n = lo;
        start = a.cu[n];
        end = a.cu[n + 1];
        if (token < start || token >= end) return;
    }
    const int64_t len = a.lengths[n];
    const bool bad = len < 0 || len > (int64_t)a.c.max_pages * a.c.page;
    if (bad && lane == 0) atomicOr(reinterpret_cast<uint32_t*>(a.ws), kCheckBadSeqlens);
    const int64_t seen = bad ? 0 : min(len, len - (end - start) + (token - start) + 1);
    const TIO* q = static_cast<const TIO*>(a.q) + token * a.qs + (int64_t)head * D + lane * V;
    float x[V], o[V], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = ld_io(q, v) * a.scale * kLog2e;
        o[v] = 0.f;
    }
    auto value = [](const uint8_t* p) {
        if constexpr (kE4m3) {
            uint32_t lo, hi;
            widen<true>(*p, lo, hi);
            return __half2float(__ushort_as_half((unsigned short)(lo & 0xffffu)));
        } else {
            return (float)(int8_t)*p;
        }
    };
    for (int64_t j = 0; j < seen; ++j) {
        const int p = a.c.table[(int64_t)n * a.c.max_pages + j / a.c.page];
        if (p < 0 || p >= a.c.num_pages) {
            if (lane == 0) atomicOr(reinterpret_cast<uint32_t*>(a.ws), kCheckBadSeqlens);
            continue;
        }
        const int64_t ph = (int64_t)p * a.Hkv + h, at = (ph * a.c.page + j % a.c.page) * D + lane * V;
        float z = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) z = fmaf(x[v], value(a.c.k + at + v), z);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
        z *= a.c.k_scale[ph];
        const float now = fmaxf(fmaxf(m, z), -3.4e38f), f = exp2f(m - now), w = exp2f(z - now), vs = a.c.v_scale[ph];
        m = now;
        l = fmaf(l, f, w);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(o[v], f, w * (value(a.c.v + at + v) * vs));
    }
    TIO* out = static_cast<TIO*>(a.out) + (token * a.Hq + head) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) st_io(out, v, l == 0.f ? 0.f : o[v] / l);
}

size_t attn_extend_workspace_bytes(int64_t, int, int, kda_dtype_t) { return 256; }

cudaError_t launch_attn_extend(const AttnExtendArgs& a, kda_dtype_t dt, cudaStream_t s)
{
    cudaError_t e = cudaMemsetAsync(a.ws, 0, 4, s);
    if (e != cudaSuccess || a.T == 0) return e;
    const int64_t ctas = (a.T * a.Hq + kWarps - 1) / kWarps;
    if (ctas > 2147483647LL) return cudaErrorInvalidValue;
    auto go = [&](auto kern) { kern<<<(unsigned)ctas, kWarps * 32, 0, s>>>(a); };
    auto by_code = [&](auto io, auto d) {
        using TIO = decltype(io);
        constexpr int D = decltype(d)::value;
        if (a.c.dtype == KDA_CACHE_E4M3) go(kda_attn_extend_kernel<TIO, D, true>);
        else go(kda_attn_extend_kernel<TIO, D, false>);
    };
    auto by_d = [&](auto io) {
        if (a.d == 32) by_code(io, std::integral_constant<int, 32>{});
        else if (a.d == 64) by_code(io, std::integral_constant<int, 64>{});
        else by_code(io, std::integral_constant<int, 128>{});
    };
    if (dt == KDA_BF16) by_d(__nv_bfloat16{});
    else by_d(float{});
    return cudaGetLastError();
}

}  // namespace kda
