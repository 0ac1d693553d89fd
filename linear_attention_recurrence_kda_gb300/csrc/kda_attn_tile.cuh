// kda_attn_tile.cuh -- which tokens a tile of the prompt kernels holds, and the rows' share of
// infinities and NaN in V.
#pragma once

#include "kda_attn.cuh"

namespace kda {

struct AttnTile {
    int64_t start;    // packed index of the sequence's first token
    int first, last;  // the tile's tokens [first, last) in the sequence; keys [0, last) are seen by some row
};

// Slots of `tokens` tokens each: sequence n owns slots cu[n] / tokens + n on, at least as many as it
// has tiles, so that a slot finds its sequence by bisection and the count needs no lengths.
inline int64_t attn_slots(const AttnArgs& a, int tokens)
{
    if (a.cu != nullptr) return a.T / tokens + a.N;
    return (a.T / a.N + tokens - 1) / tokens * a.N;
}

// The tile of a slot; false where it holds no token.  Offsets outside [0, T] are clamped.  Called by
// whole warps: 32 sequences are looked at in a step, so that a handful of sequences take one round
// of loads and not a chain of them.
__device__ __forceinline__ bool attn_tile(const AttnArgs& a, int slot, int tokens, AttnTile& t)
{
    int64_t start, end;
    int j;
    if (a.cu == nullptr) {
        const int len = (int)a.T / a.N;
        const int per = (len + tokens - 1) / tokens;
        const int n = slot / per;
        j = slot - n * per;
        start = (int64_t)n * len;
        end = start + len;
    } else {
        // the last sequence whose slots begin at or before this one
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + ((int)(threadIdx.x & 31) + 1) * step;
            const bool yes = at <= hi && a.cu[at] / tokens + at <= slot;  // below 2^31: the grid's size was checked
            lo += __popc(__ballot_sync(0xffffffffu, yes)) * step;
            hi = min(hi, lo + step - 1);
        }
        const int c0 = a.cu[lo], c1 = a.cu[lo + 1];
        j = slot - (c0 / tokens + lo);
        start = min(max((int64_t)c0, (int64_t)0), a.T);
        end = min(max((int64_t)c1, (int64_t)0), a.T);
    }
    const int64_t first = (int64_t)j * tokens;
    if (j < 0 || first >= end - start) return false;
    t.start = start;
    t.first = (int)first;
    t.last = (int)min(first + tokens, end - start);
    return true;
}

// A row's result in a channel whose first +inf, -inf and NaN stand at the given keys: every weight
// is positive, so the first that the row sees decides.
__device__ __forceinline__ float attn_odd(float x, int tok, int pinf, int ninf, int nan)
{
    if (min(min(pinf, ninf), nan) > tok) return x;
    if (nan <= tok || (pinf <= tok && ninf <= tok)) return NAN;
    return x + (pinf <= tok ? INFINITY : -INFINITY);
}

}  // namespace kda
