// kda_attn_decode.cuh -- what the kernels that read the 8-bit cache share: the workspace, the line of
// tiles that is cut among the workers, the codes' conversion.
#pragma once

#include <cuda_fp16.h>

#include "kda_attn.cuh"

namespace kda {

// Workspace: check word | per-CTA flags | records | (max, sum) of slots | outputs of slots.
// Worker w owns slots 2 w (a unit begun by an earlier worker) and 2 w + 1 (begun here).
// A call with fewer units than workers keeps its records by unit, else by the worker that began it.
struct Record {
    int32_t n, h, rt, first, last;  // unit, and the workers that hold its pieces; n < 0: none
};

struct DecodeLayout {
    size_t flags, records, ml, o, total;
};

__host__ __device__ inline DecodeLayout decode_layout(int workers, int flags, int rows, int d)
{
    DecodeLayout L;
    size_t at = 256;
    L.flags = at;
    at += ((size_t)flags * 4 + 255) / 256 * 256;
    L.records = at;
    at += ((size_t)workers * sizeof(Record) + 255) / 256 * 256;
    L.ml = at;
    at += ((size_t)workers * 2 * rows * 8 + 255) / 256 * 256;
    L.o = at;
    at += (size_t)workers * 2 * rows * d * 4;
    L.total = (at + 255) / 256 * 256;
    return L;
}

// four codes (bytes of x, low first) to two pairs of f16
template <bool kE4m3>
__device__ __forceinline__ void widen(uint32_t x, uint32_t& lo, uint32_t& hi)
{
    if constexpr (kE4m3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(x));
    } else {
        // byte b ^ 0x80 = b + 128 under the exponent of 1024 is 1024 + 128 + b; 1152 comes off exactly
        const uint32_t u = x ^ 0x80808080u;
        const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), g = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half((unsigned short)0x6480));
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&g), off);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Tokens of sequence n that count: 0 where the length is out of range.
__device__ __forceinline__ int length_of(const AttnDecodeArgs& a, int n, bool* bad = nullptr)
{
    const int len = a.lengths[n];
    const bool ok = len >= 0 && (int64_t)len <= (int64_t)a.c.max_pages * a.c.page;
    if (!ok && bad != nullptr) *bad = true;
    return ok ? len : 0;
}

template <int kTile>
__device__ __forceinline__ int tiles_of(int len)
{
    return (len + kTile - 1) / kTile;
}

// A place in the line of tiles: unit (n, h, rt) and the tile i of its `tiles`.
struct Cursor {
    int n, h, rt, i, tiles, len;
};

template <int kTile>
__device__ __forceinline__ void next_tile(const AttnDecodeArgs& a, int row_tiles, Cursor& c)
{
    if (++c.i < c.tiles) return;
    c.i = 0;
    if (++c.rt < row_tiles) return;
    c.rt = 0;
    if (++c.h < a.Hkv) return;
    c.h = 0;
    do {
        if (++c.n >= a.N) {
            c.tiles = 0;
            return;
        }
        c.len = length_of(a, c.n);
        c.tiles = tiles_of<kTile>(c.len);
    } while (c.tiles == 0);
}

// Joins the pieces that the workers of a call left in its workspace (kda_attn_decode.cu).
cudaError_t launch_attn_join(const AttnDecodeArgs& a, kda_dtype_t dt, int rows_max, int unit_rows, int workers, int flags,
                             bool by_unit, int64_t units, cudaStream_t s);

}  // namespace kda
