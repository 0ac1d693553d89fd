// kda_attn_api.cu -- C ABI of the softmax-attention operators: argument checks and launches, in the
// order of kda_api.cu (descriptor, pointers, alignment, overlap, workspace, pointer attributes).
#include <cmath>
#include <cstdint>
#include <mutex>

#include "kda_attn.cuh"
#include "kda_checks.cuh"
#include "kda_rotary.cuh"

using namespace kda::checks;

namespace {

constexpr double kMaxElems = 1099511627776.0;  // 2^40, as for the recurrence

kda_status_t check_attention(const kda_attention_t* p, bool has_q)
{
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    if (p->num_seqs < 1 || p->total_tokens < 0 || p->num_kv_heads < 1) return KDA_ERR_INVALID_ARG;
    if (p->num_kv_heads > 65535 || p->head_dim <= 0) return KDA_ERR_INVALID_ARG;
    if (p->io_dtype != KDA_F32 && p->io_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (p->q_stride < 0 || p->k_stride < 0 || p->v_stride < 0) return KDA_ERR_INVALID_ARG;
    if (has_q) {
        if (p->num_heads < 1 || p->num_heads > 65535 || p->num_heads % p->num_kv_heads != 0) return KDA_ERR_INVALID_ARG;
        if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return KDA_ERR_INVALID_ARG;
    }
    if (p->head_dim != 32 && p->head_dim != 64 && p->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    if (has_q && p->num_heads / p->num_kv_heads > kda::kMaxGroup) return KDA_ERR_UNSUPPORTED;
    const int64_t heads = has_q && p->num_heads > p->num_kv_heads ? p->num_heads : p->num_kv_heads;
    if ((double)p->total_tokens * heads * p->head_dim > kMaxElems) return KDA_ERR_UNSUPPORTED;
    if (p->total_tokens > 2147483647LL - 65536) return KDA_ERR_UNSUPPORTED;  // tile coordinates are 32-bit
    return KDA_OK;
}

// The stride between tokens in elements (0: packed), checked: a token's row fits, 16-byte steps.
kda_status_t token_stride(int64_t given, int64_t heads, const kda_attention_t& p, int64_t* out)
{
    const int64_t row = heads * p.head_dim;
    *out = given == 0 ? row : given;
    if (*out < row || (*out * (int64_t)io_size(p.io_dtype)) % 16 != 0) return KDA_ERR_INVALID_ARG;
    if ((double)p.total_tokens * (double)*out > kMaxElems) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

size_t strided_bytes(int64_t tokens, int64_t stride, int64_t row, size_t elem)
{
    return tokens > 0 ? ((size_t)(tokens - 1) * (size_t)stride + (size_t)row) * elem : 0;
}

// Tokens against the cache: whole windows, whose rows of one key head are counted in 32 bits.
kda_status_t check_windows(const kda_attention_t& p)
{
    if (p.total_tokens < p.num_seqs || p.total_tokens % p.num_seqs != 0) return KDA_ERR_INVALID_ARG;
    if (p.total_tokens / p.num_seqs * (p.num_heads / p.num_kv_heads) > 2147483647LL - 65536) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

struct CacheRanges {
    Range r[5];
};

kda_status_t check_cache(const kda_cache_t* c, const kda_attention_t& p, CacheRanges* out)
{
    if (c == nullptr) return KDA_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->max_pages < 1 || c->page_tokens < 1) return KDA_ERR_INVALID_ARG;
    if (c->dtype != KDA_CACHE_E4M3 && c->dtype != KDA_CACHE_INT8) return KDA_ERR_INVALID_ARG;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return KDA_ERR_UNSUPPORTED;
    // a sequence's tokens and a page's row are counted in 32 bits
    if ((int64_t)c->max_pages * c->page_tokens > 2147483647LL) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)c->num_pages * p.num_kv_heads > 2147483647LL) return KDA_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table) return KDA_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->block_table, 4)) return KDA_ERR_INVALID_ARG;
    const size_t ph = (size_t)c->num_pages * p.num_kv_heads;
    out->r[0] = range_of(c->k, ph * c->page_tokens * p.head_dim);
    out->r[1] = range_of(c->v, ph * c->page_tokens * p.head_dim);
    out->r[2] = range_of(c->k_scale, ph * sizeof(float));
    out->r[3] = range_of(c->v_scale, ph * sizeof(float));
    out->r[4] = range_of(c->block_table, (size_t)p.num_seqs * c->max_pages * sizeof(int32_t));
    return KDA_OK;
}

kda_status_t check_cache_pointers(const kda_cache_t& c)
{
    for (const void* ptr : {(const void*)c.k, (const void*)c.v, (const void*)c.k_scale, (const void*)c.v_scale,
                            (const void*)c.block_table}) {
        const kda_status_t st = check_device_pointer(ptr);
        if (st != KDA_OK) return st;
    }
    return KDA_OK;
}

kda::CacheArgs cache_args(const kda_cache_t& c)
{
    kda::CacheArgs a{};
    a.k = static_cast<uint8_t*>(c.k); a.v = static_cast<uint8_t*>(c.v);
    a.k_scale = c.k_scale; a.v_scale = c.v_scale; a.table = c.block_table;
    a.num_pages = c.num_pages; a.page = c.page_tokens; a.max_pages = c.max_pages; a.dtype = c.dtype;
    return a;
}

// The descriptor of a call that turns, which uses no scale.
kda_status_t check_turn_problem(const kda_attention_t* problem, bool has_q, kda_attention_t* p)
{
    if (problem == nullptr) return KDA_ERR_INVALID_ARG;
    *p = *problem;
    p->scale = 1.f;
    return check_attention(p, has_q);
}

// A part of a turn (at most a half), to the nearest multiple of 2^-64, mod 1.
uint64_t turn64(double part)
{
    const uint64_t mag = (uint64_t)std::nearbyint(std::ldexp(std::fabs(part), 64));
    return part < 0.0 ? 0 - mag : mag;
}

// The rotary descriptor, and its frequencies as fractions of a turn.
kda_status_t check_rotary(const kda_rotary_t* r, const kda_attention_t& p, bool inverse, kda::TurnArgs* out)
{
    if (r == nullptr) return KDA_ERR_INVALID_ARG;
    if (r->rot_dim < 1 || r->rot_dim > p.head_dim || r->axes < 1 || r->axes > 4) return KDA_ERR_INVALID_ARG;
    if ((r->adjacent != 0 && r->adjacent != 1) || r->reserved != 0) return KDA_ERR_INVALID_ARG;
    if (r->rot_dim % 16 != 0) return KDA_ERR_UNSUPPORTED;
    out->rot = r->rot_dim;
    out->axes = r->axes;
    out->adjacent = r->adjacent;
    out->d = p.head_dim;
    for (int i = 0; i < r->rot_dim / 2; ++i) {
        if (r->axis[i] >= r->axes || !(std::fabs(r->freq[i]) <= 65536.0)) return KDA_ERR_INVALID_ARG;
        // freq / (2 pi), with 1 / (2 pi) and the product each in two doubles: what one leaves out is taken position times
        constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
        const double hi = r->freq[i] * kHi, lo = std::fma(r->freq[i], kHi, -hi) + r->freq[i] * kLo;
        const uint64_t turn = turn64(hi - std::nearbyint(hi)) + turn64(lo);
        out->turn[i] = inverse ? 0 - turn : turn;
        out->axis[i] = r->axis[i];
    }
    return KDA_OK;
}

// One tensor that turns: its range, its output's, and where they lie (packed, or the input itself).
kda_status_t check_turned(const void* in, void* out, int64_t heads, int64_t stride, const kda_attention_t& p, int which,
                          kda::TurnRows* rows, Range* r_in, Range* r_out)
{
    rows->heads[which] = in != nullptr ? (int32_t)heads : 0;
    *r_in = *r_out = Range{0, 0};
    if ((in == nullptr) != (out == nullptr)) return KDA_ERR_INVALID_ARG;
    if (in == nullptr) return KDA_OK;
    if (!aligned(in, 16) || !aligned(out, 16)) return KDA_ERR_INVALID_ARG;
    const int64_t row = heads * p.head_dim;
    const size_t io = io_size(p.io_dtype);
    rows->in[which] = in;
    rows->out[which] = out;
    rows->in_stride[which] = stride;
    rows->out_stride[which] = in == out ? stride : row;
    *r_in = range_of(in, strided_bytes(p.total_tokens, stride, row, io));
    *r_out = in == out ? *r_in : range_of(out, (size_t)p.total_tokens * row * io);
    if (in != out && overlaps(*r_in, *r_out)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Rows of one stride that lie between one another without touching, as the views of one projection do.
bool interleaved(const void* a, size_t row_a, int64_t stride_a, const void* b, size_t row_b, int64_t stride_b, size_t io)
{
    if (stride_a != stride_b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const size_t off = x < y ? y - x : x - y, gap = (size_t)stride_a * io;
    return x < y ? off >= row_a && off + row_b <= gap : off >= row_b && off + row_a <= gap;
}

// The arguments of an append, past its descriptor.  `out`: what the call writes beside the cache (turned queries), `beside_k`, `beside_v`:
// its rows lie between those of k, of v, without touching them.
kda_status_t check_append(const void* k, const void* v, const int32_t* cu_seqlens, const int32_t* lengths, const kda_cache_t* cache,
                          const kda_attention_t& p, uint32_t* check, const Range* more_in, int more, Range out, bool beside_k, bool beside_v,
                          kda::AppendArgs& a)
{
    kda_status_t st;
    if (cu_seqlens == nullptr && p.total_tokens % p.num_seqs != 0) return KDA_ERR_INVALID_ARG;
    if ((st = token_stride(p.k_stride, p.num_kv_heads, p, &a.ks)) != KDA_OK) return st;
    if ((st = token_stride(p.v_stride, p.num_kv_heads, p, &a.vs)) != KDA_OK) return st;
    CacheRanges rc;
    if ((st = check_cache(cache, p, &rc)) != KDA_OK) return st;
    if (lengths == nullptr || (p.total_tokens > 0 && (!k || !v))) return KDA_ERR_INVALID_ARG;
    if (p.total_tokens / cache->page_tokens + 2LL * p.num_seqs > 2147483647LL) return KDA_ERR_UNSUPPORTED;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(lengths, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    if (!aligned(check, 256)) return KDA_ERR_INVALID_ARG;
    const size_t io = io_size(p.io_dtype);
    const int64_t row = (int64_t)p.num_kv_heads * p.head_dim;
    const Range in[5] = {range_of(k, strided_bytes(p.total_tokens, a.ks, row, io)),
                         range_of(v, strided_bytes(p.total_tokens, a.vs, row, io)),
                         range_of(lengths, (size_t)p.num_seqs * 4),
                         range_of(cu_seqlens, cu_seqlens ? ((size_t)p.num_seqs + 1) * 4 : 0), rc.r[4]};
    const Range rk = range_of(check, check ? 4 : 0);
    for (int i = 0; i < 4; ++i) {
        for (const Range& r : in) {
            if (overlaps(rc.r[i], r)) return KDA_ERR_INVALID_ARG;
        }
        for (int j = 0; j < i; ++j) {
            if (overlaps(rc.r[i], rc.r[j])) return KDA_ERR_INVALID_ARG;
        }
        for (int j = 0; j < more; ++j) {
            if (overlaps(rc.r[i], more_in[j])) return KDA_ERR_INVALID_ARG;
        }
        if (overlaps(rk, rc.r[i]) || overlaps(out, rc.r[i])) return KDA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 5; ++i) {
        const bool beside = i == 0 ? beside_k : i == 1 && beside_v;
        if (overlaps(rk, in[i]) || (!beside && overlaps(out, in[i]))) return KDA_ERR_INVALID_ARG;
    }
    for (int j = 0; j < more; ++j) {
        if (overlaps(rk, more_in[j])) return KDA_ERR_INVALID_ARG;
    }
    if (overlaps(rk, out)) return KDA_ERR_INVALID_ARG;
    for (const void* ptr : {k, v, (const void*)lengths, (const void*)cu_seqlens, (const void*)check}) {
        if ((st = check_device_pointer(ptr)) != KDA_OK) return st;
    }
    if ((st = check_cache_pointers(*cache)) != KDA_OK) return st;
    a.k = k; a.v = v; a.cu = cu_seqlens; a.lengths = lengths; a.check = check;
    a.T = p.total_tokens; a.N = p.num_seqs; a.Hkv = p.num_kv_heads; a.d = p.head_dim; a.c = cache_args(*cache);
    return KDA_OK;
}

}  // namespace

namespace kda {

TensorMapEncode attn_tensor_map_encoder()
{
    static TensorMapEncode fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<TensorMapEncode>(p);
        }
    });
    return fn;
}

}  // namespace kda

extern "C" {

kda_status_t kda_attention_prefill(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, void* out,
                                   const kda_attention_t* problem, void* stream)
{
    kda_status_t st = check_attention(problem, true);
    if (st != KDA_OK) return st;
    const kda_attention_t& p = *problem;
    if (cu_seqlens == nullptr && p.total_tokens % p.num_seqs != 0) return KDA_ERR_INVALID_ARG;
    kda::AttnArgs a{};
    if ((st = token_stride(p.q_stride, p.num_heads, p, &a.qs)) != KDA_OK) return st;
    if ((st = token_stride(p.k_stride, p.num_kv_heads, p, &a.ks)) != KDA_OK) return st;
    if ((st = token_stride(p.v_stride, p.num_kv_heads, p, &a.vs)) != KDA_OK) return st;
    // one CTA for each tile of tokens and key head: the grid's first axis holds 2^31 - 1
    const int group = p.num_heads / p.num_kv_heads;
    const int64_t tile = group <= 64 ? 64 / group : 1;  // tokens of the smallest tile
    if ((p.total_tokens / tile + p.num_seqs) * p.num_kv_heads > 2147483647LL) return KDA_ERR_UNSUPPORTED;
    if (p.total_tokens > 0 && (!q || !k || !v || !out)) return KDA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, v, (const void*)out}) {
        if (!aligned(ptr, 16)) return KDA_ERR_INVALID_ARG;
    }
    if (!aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    const size_t io = io_size(p.io_dtype);
    const int64_t qrow = (int64_t)p.num_heads * p.head_dim, krow = (int64_t)p.num_kv_heads * p.head_dim;
    const Range ro = range_of(out, (size_t)p.total_tokens * qrow * io);
    for (const Range& r : {range_of(q, strided_bytes(p.total_tokens, a.qs, qrow, io)),
                           range_of(k, strided_bytes(p.total_tokens, a.ks, krow, io)),
                           range_of(v, strided_bytes(p.total_tokens, a.vs, krow, io)),
                           range_of(cu_seqlens, cu_seqlens ? ((size_t)p.num_seqs + 1) * 4 : 0)}) {
        if (overlaps(ro, r)) return KDA_ERR_INVALID_ARG;
    }
    for (const void* ptr : {q, k, v, (const void*)cu_seqlens, (const void*)out}) {
        if ((st = check_device_pointer(ptr)) != KDA_OK) return st;
    }
    if (p.total_tokens == 0) return KDA_OK;
    a.q = q; a.k = k; a.v = v; a.cu = cu_seqlens; a.out = out;
    a.T = p.total_tokens; a.N = p.num_seqs; a.Hq = p.num_heads; a.Hkv = p.num_kv_heads;
    a.group = p.num_heads / p.num_kv_heads; a.d = p.head_dim; a.scale = p.scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    kda::prof_start("kda_attention_prefill", s);
    const cudaError_t e = p.io_dtype == KDA_BF16 ? kda::launch_attn_prefill_tc(a, s) : kda::launch_attn_prefill_f32(a, s);
    kda::prof_stop(s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_cache_append(const void* k, const void* v, const int32_t* cu_seqlens, const int32_t* lengths,
                              const kda_cache_t* cache, const kda_attention_t* problem, uint32_t* check, void* stream)
{
    kda_status_t st = check_attention(problem, false);
    if (st != KDA_OK) return st;
    const kda_attention_t& p = *problem;
    kda::AppendArgs a{};
    if ((st = check_append(k, v, cu_seqlens, lengths, cache, p, check, nullptr, 0, Range{0, 0}, false, false, a)) != KDA_OK) return st;
    if (p.total_tokens == 0) return KDA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    kda::prof_start("kda_cache_append", s);
    const cudaError_t e = kda::launch_cache_append(a, p.io_dtype, s);
    kda::prof_stop(s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_rotary_append(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, const int32_t* lengths,
                               const int32_t* positions, void* q_out, const kda_cache_t* cache, const kda_attention_t* problem,
                               const kda_rotary_t* rotary, uint32_t* check, void* stream)
{
    kda_attention_t p;
    kda_status_t st = check_turn_problem(problem, q != nullptr, &p);
    if (st != KDA_OK) return st;
    kda::TurnArgs t{};
    kda::TurnRows r{};
    if ((st = check_rotary(rotary, p, false, &t)) != KDA_OK) return st;
    int64_t qs = 0;
    if (q != nullptr && (st = token_stride(p.q_stride, p.num_heads, p, &qs)) != KDA_OK) return st;
    if (!aligned(positions, 4)) return KDA_ERR_INVALID_ARG;
    Range more[2], out;
    if ((st = check_turned(q, q_out, p.num_heads, qs, p, 0, &r, &more[0], &out)) != KDA_OK) return st;
    more[1] = range_of(positions, positions ? (size_t)p.total_tokens * t.axes * 4 : 0);
    if (overlaps(out, more[1])) return KDA_ERR_INVALID_ARG;
    kda::AppendArgs a{};
    // queries turned in place among the keys or values of one projection share their range, not their rows
    int64_t ks = 0, vs = 0;
    if ((st = token_stride(p.k_stride, p.num_kv_heads, p, &ks)) != KDA_OK) return st;
    if ((st = token_stride(p.v_stride, p.num_kv_heads, p, &vs)) != KDA_OK) return st;
    const size_t io = io_size(p.io_dtype), row = (size_t)p.num_heads * p.head_dim * io, krow = (size_t)p.num_kv_heads * p.head_dim * io;
    const bool place = q != nullptr && q == q_out;
    const bool beside_k = place && k != nullptr && interleaved(q, row, qs, k, krow, ks, io);
    const bool beside_v = place && v != nullptr && interleaved(q, row, qs, v, krow, vs, io);
    if ((st = check_append(k, v, cu_seqlens, lengths, cache, p, check, more, 2, out, beside_k, beside_v, a)) != KDA_OK) return st;
    for (const void* ptr : {q, (const void*)positions, (const void*)q_out}) {
        if ((st = check_device_pointer(ptr)) != KDA_OK) return st;
    }
    if (p.total_tokens == 0) return KDA_OK;
    t.positions = positions; t.cu = cu_seqlens; t.lengths = lengths; t.T = p.total_tokens; t.N = p.num_seqs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    kda::prof_start("kda_rotary_append", s);
    const cudaError_t e = kda::launch_rotary_append(a, t, r, p.io_dtype, s);
    kda::prof_stop(s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_rotary(const void* q, const void* k, const int32_t* cu_seqlens, const int32_t* lengths,
                        const int32_t* positions, void* q_out, void* k_out, const kda_attention_t* problem,
                        const kda_rotary_t* rotary, int32_t inverse, void* stream)
{
    kda_attention_t p;
    kda_status_t st = check_turn_problem(problem, q != nullptr, &p);
    if (st != KDA_OK) return st;
    if (cu_seqlens == nullptr && p.total_tokens % p.num_seqs != 0) return KDA_ERR_INVALID_ARG;
    if (inverse != 0 && inverse != 1) return KDA_ERR_INVALID_ARG;
    kda::TurnArgs t{};
    kda::TurnRows r{};
    if ((st = check_rotary(rotary, p, inverse != 0, &t)) != KDA_OK) return st;
    int64_t qs = 0, ks = 0;
    if (q != nullptr && (st = token_stride(p.q_stride, p.num_heads, p, &qs)) != KDA_OK) return st;
    if (k != nullptr && (st = token_stride(p.k_stride, p.num_kv_heads, p, &ks)) != KDA_OK) return st;
    if (p.total_tokens > 0 && q == nullptr && k == nullptr) return KDA_ERR_INVALID_ARG;
    Range in[5], out[2];
    if ((st = check_turned(q, q_out, p.num_heads, qs, p, 0, &r, &in[0], &out[0])) != KDA_OK) return st;
    if ((st = check_turned(k, k_out, p.num_kv_heads, ks, p, 1, &r, &in[1], &out[1])) != KDA_OK) return st;
    if (!aligned(cu_seqlens, 4) || !aligned(lengths, 4) || !aligned(positions, 4)) return KDA_ERR_INVALID_ARG;
    in[2] = range_of(cu_seqlens, cu_seqlens ? ((size_t)p.num_seqs + 1) * 4 : 0);
    in[3] = range_of(lengths, lengths ? (size_t)p.num_seqs * 4 : 0);
    in[4] = range_of(positions, positions ? (size_t)p.total_tokens * t.axes * 4 : 0);
    // in place, q and k may be views of one projection
    const size_t io = io_size(p.io_dtype);
    const bool both = q != nullptr && k != nullptr && q == q_out && k == k_out &&
                      interleaved(q, (size_t)p.num_heads * p.head_dim * io, qs, k, (size_t)p.num_kv_heads * p.head_dim * io, ks, io);
    for (int o = 0; o < 2; ++o) {
        for (int i = 0; i < 5; ++i) {
            if (i == o || (i < 2 && both)) continue;
            if (overlaps(out[o], in[i])) return KDA_ERR_INVALID_ARG;
        }
    }
    if (!both && overlaps(out[0], out[1])) return KDA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, (const void*)cu_seqlens, (const void*)lengths, (const void*)positions, (const void*)q_out,
                            (const void*)k_out}) {
        if ((st = check_device_pointer(ptr)) != KDA_OK) return st;
    }
    if (p.total_tokens == 0) return KDA_OK;
    t.positions = positions; t.cu = cu_seqlens; t.lengths = lengths; t.T = p.total_tokens; t.N = p.num_seqs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    kda::prof_start("kda_rotary", s);
    const cudaError_t e = kda::launch_rotary(t, r, p.io_dtype, s);
    kda::prof_stop(s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_attention_decode_workspace_bytes(const kda_attention_t* problem)
{
    if (check_attention(problem, true) != KDA_OK) return 0;
    const kda_attention_t& p = *problem;
    if (check_windows(p) != KDA_OK) return 0;
    const int64_t rows = p.total_tokens / p.num_seqs * (p.num_heads / p.num_kv_heads);
    return kda::attn_decode_workspace_bytes(rows, p.head_dim, p.io_dtype);
}

kda_status_t kda_attention_decode(const void* q, const int32_t* lengths, const kda_cache_t* cache, void* out,
                                  const kda_attention_t* problem, void* workspace, size_t workspace_bytes, void* stream)
{
    kda_status_t st = check_attention(problem, true);
    if (st != KDA_OK) return st;
    const kda_attention_t& p = *problem;
    if ((st = check_windows(p)) != KDA_OK) return st;
    kda::AttnDecodeArgs a{};
    if ((st = token_stride(p.q_stride, p.num_heads, p, &a.qs)) != KDA_OK) return st;
    CacheRanges rc;
    if ((st = check_cache(cache, p, &rc)) != KDA_OK) return st;
    if (!q || !lengths || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lengths, 4)) return KDA_ERR_INVALID_ARG;
    const size_t io = io_size(p.io_dtype);
    const int64_t row = (int64_t)p.num_heads * p.head_dim;
    const Range rq = range_of(q, strided_bytes(p.total_tokens, a.qs, row, io));
    const Range rl = range_of(lengths, (size_t)p.num_seqs * 4);
    const Range ro = range_of(out, (size_t)p.total_tokens * row * io);
    const size_t need = kda_attention_decode_workspace_bytes(problem);
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const Range rw = range_of(workspace, need);
    if (overlaps(ro, rq) || overlaps(ro, rl) || overlaps(rw, rq) || overlaps(rw, rl) || overlaps(rw, ro))
        return KDA_ERR_INVALID_ARG;
    for (const Range& r : rc.r) {
        if (overlaps(ro, r) || overlaps(rw, r)) return KDA_ERR_INVALID_ARG;
    }
    for (const void* ptr : {q, (const void*)lengths, (const void*)out, (const void*)workspace}) {
        if ((st = check_device_pointer(ptr)) != KDA_OK) return st;
    }
    if ((st = check_cache_pointers(*cache)) != KDA_OK) return st;
    a.q = q; a.lengths = lengths; a.out = out; a.ws = static_cast<unsigned char*>(workspace);
    a.N = p.num_seqs; a.L = (int32_t)(p.total_tokens / p.num_seqs); a.Hq = p.num_heads; a.Hkv = p.num_kv_heads;
    a.group = p.num_heads / p.num_kv_heads; a.d = p.head_dim; a.scale = p.scale; a.c = cache_args(*cache);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    kda::prof_start("kda_attention_decode", s);
    const cudaError_t e = kda::launch_attn_decode(a, p.io_dtype, s);
    kda::prof_stop(s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_attention_extend_workspace_bytes(const kda_attention_t* problem)
{
    if (check_attention(problem, true) != KDA_OK) return 0;
    const kda_attention_t& p = *problem;
    return kda::attn_extend_workspace_bytes(p.total_tokens, p.num_heads / p.num_kv_heads, p.head_dim, p.io_dtype);
}

kda_status_t kda_attention_extend(const void* q, const int32_t* cu_seqlens, const int32_t* lengths, const kda_cache_t* cache,
                                  void* out, const kda_attention_t* problem, void* workspace, size_t workspace_bytes,
                                  void* stream)
{
    kda_status_t st = check_attention(problem, true);
    if (st != KDA_OK) return st;
    const kda_attention_t& p = *problem;
    if (cu_seqlens == nullptr && p.total_tokens % p.num_seqs != 0) return KDA_ERR_INVALID_ARG;
    kda::AttnExtendArgs a{};
    if ((st = token_stride(p.q_stride, p.num_heads, p, &a.qs)) != KDA_OK) return st;
    CacheRanges rc;
    if ((st = check_cache(cache, p, &rc)) != KDA_OK) return st;
    if (lengths == nullptr || (p.total_tokens > 0 && (!q || !out))) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lengths, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    const size_t io = io_size(p.io_dtype);
    const int64_t row = (int64_t)p.num_heads * p.head_dim;
    const Range rq = range_of(q, strided_bytes(p.total_tokens, a.qs, row, io));
    const Range rl = range_of(lengths, (size_t)p.num_seqs * 4);
    const Range ru = range_of(cu_seqlens, cu_seqlens ? ((size_t)p.num_seqs + 1) * 4 : 0);
    const Range ro = range_of(out, (size_t)p.total_tokens * row * io);
    const size_t need = kda_attention_extend_workspace_bytes(problem);
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const Range rw = range_of(workspace, need);
    for (const Range& r : {rq, rl, ru, rc.r[0], rc.r[1], rc.r[2], rc.r[3], rc.r[4]}) {
        if (overlaps(ro, r) || overlaps(rw, r)) return KDA_ERR_INVALID_ARG;
    }
    if (overlaps(rw, ro)) return KDA_ERR_INVALID_ARG;
    for (const void* ptr : {q, (const void*)cu_seqlens, (const void*)lengths, (const void*)out, (const void*)workspace}) {
        if ((st = check_device_pointer(ptr)) != KDA_OK) return st;
    }
    if ((st = check_cache_pointers(*cache)) != KDA_OK) return st;
    a.q = q; a.cu = cu_seqlens; a.lengths = lengths; a.out = out; a.ws = static_cast<unsigned char*>(workspace);
    a.T = p.total_tokens; a.N = p.num_seqs; a.Hq = p.num_heads; a.Hkv = p.num_kv_heads;
    a.group = p.num_heads / p.num_kv_heads; a.d = p.head_dim; a.scale = p.scale; a.c = cache_args(*cache);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    kda::prof_start("kda_attention_extend", s);
    const cudaError_t e = kda::launch_attn_extend(a, p.io_dtype, s);
    kda::prof_stop(s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
