// kda_attn.cuh -- arguments and launchers of the softmax-attention kernels (declared in kda.h):
// prompts (kda_attn_prefill_tc.cu for bf16, kda_attn_prefill_f32.cu), the 8-bit paged cache (kda_cache.cu) and
// the tokens that read it (kda_attn_decode.cu).
#pragma once

#include <atomic>

#include <cuda.h>

#include "kda_internal.cuh"

namespace kda {

constexpr int kMaxGroup = 128;  // query heads that may share a key head: a tile's rows

struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* cu;  // NULL: N equal lengths
    void* out;
    int64_t T;
    int64_t qs, ks, vs;  // elements between tokens
    int32_t N, Hq, Hkv, group, d;
    float scale;
};

struct CacheArgs {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    const int32_t* table;
    int32_t num_pages, page, max_pages;
    kda_cache_dtype_t dtype;
};

struct AppendArgs {
    const void* k;
    const void* v;
    const int32_t* cu;       // NULL: T / N new tokens each
    const int32_t* lengths;  // with the new tokens
    uint32_t* check;         // NULL, or a word whose kCheckBadSeqlens bit is set on a bad length or page
    int64_t T, ks, vs;
    int32_t N, Hkv, d;
    CacheArgs c;
};

struct AttnDecodeArgs {
    const void* q;
    const int32_t* lengths;
    void* out;
    unsigned char* ws;
    int64_t qs;
    int32_t N, L, Hq, Hkv, group, d;
    float scale;
    CacheArgs c;
};

struct AttnExtendArgs {
    const void* q;
    const int32_t* cu;       // NULL: T / N new tokens each
    const int32_t* lengths;  // with the new tokens
    void* out;
    unsigned char* ws;
    int64_t T, qs;
    int32_t N, Hq, Hkv, group, d;
    float scale;
    CacheArgs c;
};

cudaError_t launch_attn_prefill_f32(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_prefill_tc(const AttnArgs& a, cudaStream_t s);  // bf16
cudaError_t launch_cache_append(const AppendArgs& a, kda_dtype_t dt, cudaStream_t s);
cudaError_t launch_attn_decode(const AttnDecodeArgs& a, kda_dtype_t dt, cudaStream_t s);
size_t attn_decode_workspace_bytes(int64_t rows, int d, kda_dtype_t dt);  // rows: window x group

cudaError_t launch_attn_extend(const AttnExtendArgs& a, kda_dtype_t dt, cudaStream_t s);
size_t attn_extend_workspace_bytes(int64_t tokens, int group, int d, kda_dtype_t dt);

// The form for many rows a key head (kda_attn_window.cu): does it take a call, what does it need.
bool attn_window_takes(int64_t rows, int d, kda_dtype_t dt, int64_t capacity);  // keys that a sequence's pages hold
size_t attn_window_workspace_bytes(int64_t rows, int d);
cudaError_t launch_attn_window(const AttnDecodeArgs& a, cudaStream_t s);

// A kernel's dynamic shared memory limit, raised once for each device (the call costs about half a
// microsecond, which short calls feel).
struct SmemLimit {
    std::atomic<uint64_t> done{0};
    template <typename F>
    cudaError_t raise(F* kernel, int bytes)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
        if (bit != 0 && (done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

// cuTensorMapEncodeTiled of the loaded driver, or NULL (kda_attn_api.cu).
using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncode attn_tensor_map_encoder();

}  // namespace kda
