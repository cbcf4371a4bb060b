// k_cache.cu -- the paged key-value cache: writing new tokens or a tree's accepted
// path into pages (bf16, or quantised to e4m3 as it is written), and reading pages
// back into the contiguous cache of the tree-masked attention, sm_100a.
//
// Every row is 128 values of one (token, key/value head): 16 lanes hold it, 8 values (16
// bytes) each, take the largest magnitude by four shuffles and store 8 bytes each.  Nothing is
// reused, so the kernels are bound by HBM, and a thread's chain of look-ups (sequence, page)
// has to be paid by enough data: 16 lanes take four heads of a token, keys and values, eight
// independent 16-byte loads in flight for each thread (8192 tokens of 8 heads written to e4m3
// pages and read back, 101 MB: 24.9 us; with a head at a time 30.1).
#include "seq_pages.cuh"

namespace stree {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsPerUnit = 4;               // heads of a token that 16 lanes take
constexpr int kUnitsPerBlock = kThreads / 16;

struct CacheArgs {
    const uint16_t *k, *v;                     // packed rows (write, commit)
    uint16_t *k_ctx, *v_ctx;                   // contiguous cache (read)
    uint8_t *k_pages, *v_pages, *k_scales, *v_scales;
    const int32_t *cu, *start, *path, *path_len, *lens, *table;
    int32_t *err;
    int total, batch, n_nodes, maxlen, ctx_cap, heads, n_pages, page_size, max_pages;
};

enum Mode { kWrite, kCommit, kRead };

// Binary search in the packed offsets for the sequence of row t (verified by the caller).
__device__ __forceinline__ int seq_of_row(const int32_t *cu, int batch, int t)
{
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// 8 values of a row, written into its page slot; the row's 16 lanes call it together.
template <bool kE4m3>
__device__ __forceinline__ void put(const uint4 &x, uint8_t *pages, uint8_t *scales, size_t slot, int l16, uint32_t mask)
{
    if (!kE4m3) {
        *reinterpret_cast<uint4 *>(pages + slot * (kCacheDim * 2) + l16 * 16) = x;
        return;
    }
    uint32_t top = max(max(finite_top2(x.x), finite_top2(x.y)), max(finite_top2(x.z), finite_top2(x.w)));
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) top = max(top, __shfl_xor_sync(mask, top, d));
    const uint32_t s = scale_of_top(top);
    const float inv = power_of_two(254u - s);
    uint2 r;
    r.x = quantise2(x.x, inv) | (quantise2(x.y, inv) << 16);
    r.y = quantise2(x.z, inv) | (quantise2(x.w, inv) << 16);
    *reinterpret_cast<uint2 *>(pages + slot * kCacheDim + l16 * 8) = r;
    if (l16 == 0) scales[slot] = (uint8_t)s;
}

// 8 values of a page slot as they lie there (the scale beside them), and as bf16.
struct Held {
    uint4 x;
    uint32_t scale;
};

template <bool kE4m3>
__device__ __forceinline__ Held take(const uint8_t *pages, const uint8_t *scales, size_t slot, int l16)
{
    Held h{};
    if (kE4m3) {
        const uint2 r = __ldcs(reinterpret_cast<const uint2 *>(pages + slot * kCacheDim + l16 * 8));
        h.x.x = r.x;
        h.x.y = r.y;
        h.scale = __ldg(scales + slot);
    } else {
        h.x = __ldcs(reinterpret_cast<const uint4 *>(pages + slot * (kCacheDim * 2) + l16 * 16));
    }
    return h;
}

template <bool kE4m3>
__device__ __forceinline__ uint4 values(const Held &h)
{
    if (!kE4m3) return h.x;
    const float s = power_of_two(h.scale);
    return make_uint4(dequantise2(h.x.x & 0xffffu, s), dequantise2(h.x.x >> 16, s), dequantise2(h.x.y & 0xffffu, s),
                      dequantise2(h.x.y >> 16, s));
}

template <Mode kMode, bool kE4m3>
__global__ void __launch_bounds__(kThreads) cache_kernel(const CacheArgs a)
{
    pdl_start();
    if (blockIdx.x == gridDim.x - 1) {         // the error word
        PageCheck c{};
        c.cu = kMode == kWrite ? a.cu : nullptr;
        c.count = kMode == kCommit ? a.path_len : a.lens;
        c.start = kMode == kRead ? nullptr : a.start;
        c.table = a.table;
        c.batch = a.batch;
        c.total = a.total;
        c.n_pages = a.n_pages;
        c.page_size = a.page_size;
        c.max_pages = a.max_pages;
        c.clamp = kMode == kRead ? a.ctx_cap : kMode == kCommit ? a.maxlen : -1;
        check_pages(c, a.err);
        if (kMode == kCommit && a.err)
            for (int i = threadIdx.x; i < a.batch * a.maxlen; i += kThreads) {
                const int b = i / a.maxlen, j = i % a.maxlen;
                if (j >= __ldg(a.path_len + b)) continue;
                const int node = __ldg(a.path + i);
                if (node < 0 || node >= a.n_nodes) latch_error(a.err, STREE_ERR_BAD_PATH, b, j, node);
            }
        return;
    }
    const int l16 = threadIdx.x & 15;
    const uint32_t mask = threadIdx.x & 16 ? 0xffff0000u : 0x0000ffffu;
    const uint32_t unit = blockIdx.x * kUnitsPerBlock + (threadIdx.x >> 4);   // below 2^31 (checked on the host)
    const uint32_t per_tok = (a.heads + kHeadsPerUnit - 1) / kHeadsPerUnit;
    const int tok = (int)(unit / per_tok), h0 = (int)(unit % per_tok) * kHeadsPerUnit;
    int b, pos;
    size_t src;                                // token row of k / v, or of k_ctx / v_ctx
    if (kMode == kWrite) {
        if (tok >= a.total) return;
        b = seq_of_row(a.cu, a.batch, tok);
        const int2 r = seq_range(a.cu, b, a.total);
        if (tok < r.x || tok >= r.y) return;   // behind the last sequence
        const int at = __ldg(a.start + b);
        if (at < 0 || (long long)at + (r.y - r.x) > (long long)a.max_pages * a.page_size) return;
        pos = tok - r.x + at;
        src = (size_t)tok;
    } else if (kMode == kCommit) {
        b = tok / a.maxlen;
        if (b >= a.batch) return;
        const int j = tok % a.maxlen, n = min(max(__ldg(a.path_len + b), 0), a.maxlen);
        if (j >= n) return;
        const int node = __ldg(a.path + tok), at = __ldg(a.start + b);
        if (node < 0 || node >= a.n_nodes || at < 0 || (long long)at + n > (long long)a.max_pages * a.page_size) return;
        pos = at + j;
        src = (size_t)b * a.n_nodes + node;
    } else {
        b = tok / a.ctx_cap;
        if (b >= a.batch) return;
        pos = tok % a.ctx_cap;
        if (pos >= min((long long)__ldg(a.lens + b), (long long)a.max_pages * a.page_size)) return;
        src = (size_t)tok;
    }
    const int page = __ldg(a.table + (size_t)b * a.max_pages + pos / a.page_size);
    if (page < 0 || page >= a.n_pages) return;
    const size_t slot0 = ((size_t)page * a.heads + h0) * a.page_size + pos % a.page_size;
    const size_t row0 = (src * a.heads + h0) * kCacheDim + l16 * 8;
    const int n = min(kHeadsPerUnit, a.heads - h0);
    if (kMode == kRead) {
        Held k[kHeadsPerUnit], v[kHeadsPerUnit];
#pragma unroll
        for (int h = 0; h < kHeadsPerUnit; ++h)
            if (h < n) {
                k[h] = take<kE4m3>(a.k_pages, a.k_scales, slot0 + (size_t)h * a.page_size, l16);
                v[h] = take<kE4m3>(a.v_pages, a.v_scales, slot0 + (size_t)h * a.page_size, l16);
            }
#pragma unroll
        for (int h = 0; h < kHeadsPerUnit; ++h)
            if (h < n) {
                *reinterpret_cast<uint4 *>(a.k_ctx + row0 + h * kCacheDim) = values<kE4m3>(k[h]);
                *reinterpret_cast<uint4 *>(a.v_ctx + row0 + h * kCacheDim) = values<kE4m3>(v[h]);
            }
    } else {
        uint4 k[kHeadsPerUnit], v[kHeadsPerUnit];
#pragma unroll
        for (int h = 0; h < kHeadsPerUnit; ++h)
            if (h < n) {
                k[h] = __ldcs(reinterpret_cast<const uint4 *>(a.k + row0 + h * kCacheDim));
                v[h] = __ldcs(reinterpret_cast<const uint4 *>(a.v + row0 + h * kCacheDim));
            }
#pragma unroll
        for (int h = 0; h < kHeadsPerUnit; ++h)
            if (h < n) {                       // the same for a unit's 16 lanes
                put<kE4m3>(k[h], a.k_pages, a.k_scales, slot0 + (size_t)h * a.page_size, l16, mask);
                put<kE4m3>(v[h], a.v_pages, a.v_scales, slot0 + (size_t)h * a.page_size, l16, mask);
            }
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Tokens to cover -> blocks, one more for the error word.
template <Mode kMode>
stree_status launch_cache(const CacheArgs &a, stree_dtype cache, long long tokens, void *stream)
{
    const long long units = tokens * ((a.heads + kHeadsPerUnit - 1) / kHeadsPerUnit);
    if (units > 0x7fffff00LL) return STREE_ERR_UNSUPPORTED;
    const long long blocks = (units + kUnitsPerBlock - 1) / kUnitsPerBlock + 1;
    const cudaError_t e = launch_pdl(cache == STREE_E4M3 ? cache_kernel<kMode, true> : cache_kernel<kMode, false>,
                                     dim3((unsigned)blocks), kThreads, 0, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? STREE_OK : STREE_ERR_CUDA;
}

}  // namespace

// Shape and pointer checks shared by every call that takes a paged cache.
stree_status check_cache(const void *k_pages, const void *v_pages, const void *k_scales, const void *v_scales,
                         const int32_t *table, int batch, int heads_kv, int head_dim, int n_pages, int page_size,
                         int max_pages, stree_dtype cache)
{
    if (batch < 0 || heads_kv < 1 || head_dim != kCacheDim || n_pages < 1 || max_pages < 1 || page_size < 8 ||
        page_size > 4096 || page_size % 8 != 0 || (cache != STREE_BF16 && cache != STREE_E4M3))
        return STREE_ERR_UNSUPPORTED;
    // Positions and page rows are 32-bit numbers inside the kernels (byte offsets are not).
    if ((long long)n_pages * page_size * heads_kv > 0x7fffffffLL || (long long)max_pages * page_size > 0x40000000LL)
        return STREE_ERR_UNSUPPORTED;
    if (batch == 0) return STREE_OK;
    if (!k_pages || !v_pages || !table || (cache == STREE_E4M3) != (k_scales != nullptr) ||
        (cache == STREE_E4M3) != (v_scales != nullptr))
        return STREE_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_scales) || !aligned16(v_scales) || !aligned4(table))
        return STREE_ERR_MISALIGNED;
    return STREE_OK;
}

}  // namespace stree

using namespace stree;

extern "C" stree_status stree_cache_write(const void *k, const void *v, const int32_t *cu_seqlens,
                                          const int32_t *start, const int32_t *page_table, int total, int batch,
                                          int heads_kv, int head_dim, int n_pages, int page_size, int max_pages,
                                          stree_dtype dtype, stree_dtype cache_dtype, void *k_pages, void *v_pages,
                                          uint8_t *k_scales, uint8_t *v_scales, int32_t *err_out, void *stream)
{
    stree_status st = check_cache(k_pages, v_pages, k_scales, v_scales, page_table, batch, heads_kv, head_dim, n_pages,
                                  page_size, max_pages, cache_dtype);
    if (st != STREE_OK) return st;
    if (total < 0 || dtype != STREE_BF16) return STREE_ERR_UNSUPPORTED;
    if (batch == 0) return STREE_OK;
    if (!cu_seqlens || !start || (total > 0 && (!k || !v))) return STREE_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned4(cu_seqlens) || !aligned4(start) || !aligned4(err_out))
        return STREE_ERR_MISALIGNED;
    CacheArgs a{};
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.cu = cu_seqlens;
    a.start = start;
    a.table = page_table;
    a.k_pages = static_cast<uint8_t *>(k_pages);
    a.v_pages = static_cast<uint8_t *>(v_pages);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.err = err_out;
    a.total = total;
    a.batch = batch;
    a.heads = heads_kv;
    a.n_pages = n_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    return launch_cache<kWrite>(a, cache_dtype, total, stream);
}

extern "C" stree_status stree_cache_commit(const void *k_tree, const void *v_tree, const int32_t *accepted_path,
                                           const int32_t *path_len, int maxlen, const int32_t *start,
                                           const int32_t *page_table, int n_nodes, int batch, int heads_kv,
                                           int head_dim, int n_pages, int page_size, int max_pages, stree_dtype dtype,
                                           stree_dtype cache_dtype, void *k_pages, void *v_pages, uint8_t *k_scales,
                                           uint8_t *v_scales, int32_t *err_out, void *stream)
{
    stree_status st = check_cache(k_pages, v_pages, k_scales, v_scales, page_table, batch, heads_kv, head_dim, n_pages,
                                  page_size, max_pages, cache_dtype);
    if (st != STREE_OK) return st;
    if (n_nodes < 1 || n_nodes > kMaxNodes || maxlen < 1 || maxlen > kMaxNodes || dtype != STREE_BF16)
        return STREE_ERR_UNSUPPORTED;
    if ((long long)batch * maxlen > 0x7fffffffLL) return STREE_ERR_UNSUPPORTED;
    if (batch == 0) return STREE_OK;
    if (!k_tree || !v_tree || !accepted_path || !path_len || !start) return STREE_ERR_INVALID_ARG;
    if (!aligned16(k_tree) || !aligned16(v_tree) || !aligned4(accepted_path) || !aligned4(path_len) ||
        !aligned4(start) || !aligned4(err_out))
        return STREE_ERR_MISALIGNED;
    CacheArgs a{};
    a.k = static_cast<const uint16_t *>(k_tree);
    a.v = static_cast<const uint16_t *>(v_tree);
    a.path = accepted_path;
    a.path_len = path_len;
    a.start = start;
    a.table = page_table;
    a.k_pages = static_cast<uint8_t *>(k_pages);
    a.v_pages = static_cast<uint8_t *>(v_pages);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.err = err_out;
    a.batch = batch;
    a.n_nodes = n_nodes;
    a.maxlen = maxlen;
    a.heads = heads_kv;
    a.n_pages = n_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    return launch_cache<kCommit>(a, cache_dtype, (long long)batch * maxlen, stream);
}

extern "C" stree_status stree_cache_read(const void *k_pages, const void *v_pages, const uint8_t *k_scales,
                                         const uint8_t *v_scales, const int32_t *page_table, const int32_t *seq_len,
                                         int batch, int ctx_cap, int heads_kv, int head_dim, int n_pages, int page_size,
                                         int max_pages, stree_dtype cache_dtype, stree_dtype dtype, void *k_ctx,
                                         void *v_ctx, int32_t *err_out, void *stream)
{
    stree_status st = check_cache(k_pages, v_pages, k_scales, v_scales, page_table, batch, heads_kv, head_dim, n_pages,
                                  page_size, max_pages, cache_dtype);
    if (st != STREE_OK) return st;
    if (ctx_cap < 0 || dtype != STREE_BF16) return STREE_ERR_UNSUPPORTED;
    if (batch == 0) return STREE_OK;
    if (!seq_len || (ctx_cap > 0 && (!k_ctx || !v_ctx))) return STREE_ERR_INVALID_ARG;
    if (!aligned16(k_ctx) || !aligned16(v_ctx) || !aligned4(seq_len) || !aligned4(err_out)) return STREE_ERR_MISALIGNED;
    CacheArgs a{};
    a.k_ctx = static_cast<uint16_t *>(k_ctx);
    a.v_ctx = static_cast<uint16_t *>(v_ctx);
    a.lens = seq_len;
    a.table = page_table;
    a.k_pages = static_cast<uint8_t *>(const_cast<void *>(k_pages));
    a.v_pages = static_cast<uint8_t *>(const_cast<void *>(v_pages));
    a.k_scales = const_cast<uint8_t *>(k_scales);
    a.v_scales = const_cast<uint8_t *>(v_scales);
    a.err = err_out;
    a.batch = batch;
    a.ctx_cap = ctx_cap;
    a.heads = heads_kv;
    a.n_pages = n_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    return launch_cache<kRead>(a, cache_dtype, (long long)batch * ctx_cap, stream);
}
