// kda_rotary.cuh -- rotary positions: angles as fractions of a turn, which tokens stand where, and the turning of rows of
// heads (kda_rotary.cu; kda_cache.cu turns keys on their way into the cache).
//
// A position p times a frequency f is an angle of p f / (2 pi) turns, of which only the fraction counts.  f / (2 pi) mod 1 is kept
// as a 64-bit fraction F, off by at most 2^-64, and the integer product p F mod 2^64 is exact: p takes that to 2^-33 of a turn at
// most, and of the product the upper 32 bits, which leave 2^-32, go on.
#pragma once

#include "kda_attn.cuh"

namespace kda {

constexpr int kMaxPairs = 64;

struct TurnArgs {
    uint64_t turn[kMaxPairs];  // of a pair's frequency, as a fraction of a turn
    uint8_t axis[kMaxPairs];
    const int32_t* positions;  // [axes][T], or NULL
    const int32_t* cu;         // NULL: N equal lengths
    const int32_t* lengths;    // NULL: sequences begin with these tokens
    int64_t T;
    int32_t N, rot, axes, adjacent, d;
};

// Rows of heads that turn: q's, then k's.
struct TurnRows {
    const void* in[2];
    void* out[2];
    int64_t in_stride[2], out_stride[2];  // elements between tokens
    int32_t heads[2];
    int32_t per_task;  // heads that a warp takes of its tokens
};

// sin and cos of a 32-bit fraction of a turn: the nearest quarter comes off as an integer, what is left is within an
// eighth of a turn and exact to fp32's relative precision.
__device__ __forceinline__ void sincos_turn(uint32_t x, float& s, float& c)
{
    const uint32_t quarter = (x + 0x20000000u) >> 30;
    const int rest = (int)(x - (quarter << 30));
    float a, b;
    sincospif((float)rest * 0x1p-31f, &a, &b);
    const float u = quarter & 1u ? b : a, v = quarter & 1u ? a : b;
    s = quarter & 2u ? -u : u;
    c = ((quarter + 1u) & 2u) ? -v : v;
}

__device__ __forceinline__ void sincos_of(const TurnArgs& t, int pair, int position, float& s, float& c)
{
    sincos_turn((uint32_t)((t.turn[pair] * (uint64_t)(int64_t)position) >> 32), s, c);
}

// The task of a warp: the tokens [task / groups * per, + per) with per = 512 / d, and a group of heads.  A lane has a token
// and two vectors of eight channels of each of its heads: pairs (i, i + rot / 2) lie in the vectors i and i + rot / 16,
// adjacent ones in one vector.  Sines and cosines are formed once and serve all of the lane's heads.
// All 32 lanes come here.
template <typename TIO>
__device__ __forceinline__ void turn_task(const TurnArgs& t, const TurnRows& r, int64_t task, int groups)
{
    const int lane = threadIdx.x & 31;
    const int per_token = t.d >> 4;  // lanes of a token: 2, 4 or 8
    const int per = 32 / per_token;
    const int64_t first = task / groups * per;
    const int h0 = (int)(task % groups) * r.per_task;
    const int64_t token = first + lane / per_token;
    const int part = lane % per_token;
    bool on = token < t.T;
    int place = 0;  // in its sequence
    if (t.cu != nullptr) {
        if (t.positions != nullptr) {
            on = on && token < t.cu[t.N];
        } else {
            // the last sequence that begins at or before the first token, 32 looked at in a step; then the boundaries
            // behind it that each token has passed
            int lo = 0, hi = t.N - 1;
            while (lo < hi) {
                const int step = (hi - lo + 31) / 32;
                const int at = lo + (lane + 1) * step;
                const bool yes = at <= hi && t.cu[at] <= first;
                lo += __popc(__ballot_sync(0xffffffffu, yes)) * step;
                hi = min(hi, lo + step - 1);
            }
            int n = lo;
            for (;;) {
                const int at = lo + 1 + lane;
                const int64_t bound = at <= t.N ? t.cu[at] : INT64_MAX;
                int past = 0;
                for (int i = 0; i < per; ++i) {
                    const int c = __popc(__ballot_sync(0xffffffffu, bound <= first + i));
                    if (lane / per_token == i) past = c;
                }
                if (n == lo) n += past;
                if (!__any_sync(0xffffffffu, past == 32 && n == lo + 32)) break;
                lo += 32;
            }
            on = on && n < t.N;
            if (on) {
                const int c0 = t.cu[n];
                on = c0 >= 0 && token >= c0;
                place = (int)(token - c0);
                if (t.lengths != nullptr) place += t.lengths[n] - (t.cu[n + 1] - c0);
            }
        }
    } else if (t.positions == nullptr && on) {
        const int count = (int)(t.T / t.N), n = (int)(token / count);
        place = (int)(token - (int64_t)n * count);
        if (t.lengths != nullptr) place += t.lengths[n] - count;
    }
    if (!on) return;  // (no collective operation follows)
    // the lane's vectors of a head, as channels, and the pair of each pair of values
    const bool turns = t.adjacent || part < (t.rot >> 4);
    const int half = t.rot >> 1;
    int c0, c1;
    if (t.adjacent) {
        c0 = 8 * part;
        c1 = c0 + (t.d >> 1);
    } else if (turns) {
        c0 = 8 * part;
        c1 = c0 + half;
    } else {
        c0 = t.rot + 16 * (part - (t.rot >> 4));
        c1 = c0 + 8;
    }
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = t.adjacent ? (i < 4 ? (c0 >> 1) + i : (c1 >> 1) + i - 4) : c0 + i;
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (turns && pair < half) {
            const int p = t.positions != nullptr ? t.positions[(int64_t)t.axis[pair] * t.T + token] : place;
            sincos_of(t, pair, p, sn[i], cs[i]);
        }
    }
    // adjacent vectors past rot hold no pair: copied as they are (a turn by nothing could change a NaN's bits or a zero's sign)
    const bool turn0 = turns && (!t.adjacent || c0 < t.rot), turn1 = turns && (!t.adjacent || c1 < t.rot);
    constexpr int W = sizeof(TIO) / 2;  // 16-byte words of a vector
    constexpr int kAhead = sizeof(TIO) == 2 ? 4 : 2;
    const int all = r.heads[0] + r.heads[1], h1 = min(all, h0 + r.per_task);
    auto place_of = [&](int h, const TIO*& src, TIO*& dst) {
        const int x = h < r.heads[0] ? 0 : 1, y = x ? h - r.heads[0] : h;
        src = static_cast<const TIO*>(r.in[x]) + token * r.in_stride[x] + (int64_t)y * t.d;
        dst = static_cast<TIO*>(r.out[x]) + token * r.out_stride[x] + (int64_t)y * t.d;
    };
    for (int h = h0; h < h1; h += kAhead) {
        uint4 u[kAhead][2][W];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (h + e >= h1) continue;
            const TIO* src;
            TIO* dst;
            place_of(h + e, src, dst);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                u[e][0][w] = reinterpret_cast<const uint4*>(src + c0)[w];
                u[e][1][w] = reinterpret_cast<const uint4*>(src + c1)[w];
            }
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (h + e >= h1) continue;
            const TIO* src;
            TIO* dst;
            place_of(h + e, src, dst);
            float x[2][8], y[2][8];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if constexpr (W == 1) {
                    const uint32_t q[4] = {u[e][v][0].x, u[e][v][0].y, u[e][v][0].z, u[e][v][0].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[v][2 * i] = __uint_as_float(q[i] << 16);
                        x[v][2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        x[v][4 * w] = __uint_as_float(u[e][v][w].x);
                        x[v][4 * w + 1] = __uint_as_float(u[e][v][w].y);
                        x[v][4 * w + 2] = __uint_as_float(u[e][v][w].z);
                        x[v][4 * w + 3] = __uint_as_float(u[e][v][w].w);
                    }
                }
            }
            if (t.adjacent) {
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float c = cs[4 * v + i], s = sn[4 * v + i];
                        y[v][2 * i] = fmaf(x[v][2 * i], c, -x[v][2 * i + 1] * s);
                        y[v][2 * i + 1] = fmaf(x[v][2 * i + 1], c, x[v][2 * i] * s);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[0][i] = fmaf(x[0][i], cs[i], -x[1][i] * sn[i]);
                    y[1][i] = fmaf(x[1][i], cs[i], x[0][i] * sn[i]);
                }
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const bool turned = v ? turn1 : turn0;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint4 z;
                    if constexpr (W == 1) {
                        uint32_t q[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(y[v][2 * i], y[v][2 * i + 1]);
                            q[i] = *reinterpret_cast<const uint32_t*>(&b);
                        }
                        z = make_uint4(q[0], q[1], q[2], q[3]);
                    } else {
                        z = make_uint4(__float_as_uint(y[v][4 * w]), __float_as_uint(y[v][4 * w + 1]),
                                       __float_as_uint(y[v][4 * w + 2]), __float_as_uint(y[v][4 * w + 3]));
                    }
                    reinterpret_cast<uint4*>(dst + (v ? c1 : c0))[w] = turned ? z : u[e][v][w];
                }
            }
        }
    }
}

// Warps that a call's rows take: tokens by groups of heads.  Few tokens are spread over so many groups that about twelve
// warps an SM are at work, which the registers let it hold at a time; with many a warp keeps its tokens' sines for all
// heads.  Measured with 8, 12, 16 and 32 warps wanted: 1000 tokens of 40 heads of 128 channels 6.6, 5.6, 7.7, 9.6 us; 5000
// tokens 23.0, 21.1, 21.0, 23.0; 9000 of 20 heads 13.5, 13.5, 16.4, 18.7; 20,000 tokens 78 with all.
inline int64_t turn_tasks(const TurnArgs& t, TurnRows& r, int* groups)
{
    const int all = r.heads[0] + r.heads[1], per = 512 / t.d;
    const int64_t tokens = (t.T + per - 1) / per;
    const int64_t want = (int64_t)sm_count_of_current_device() * 12;
    int64_t g = tokens > 0 ? (want + tokens - 1) / tokens : 1;
    if (g > all) g = all;
    r.per_task = (int)((all + g - 1) / g);
    *groups = (all + r.per_task - 1) / r.per_task;
    return tokens * *groups;
}

cudaError_t launch_rotary(const TurnArgs& t, const TurnRows& r, kda_dtype_t dt, cudaStream_t s);
// kda_cache.cu: keys turned on the way; q's rows (heads[0] = 0: none) in the same launch
cudaError_t launch_rotary_append(const AppendArgs& a, const TurnArgs& t, const TurnRows& q, kda_dtype_t dt, cudaStream_t s);

}  // namespace kda
