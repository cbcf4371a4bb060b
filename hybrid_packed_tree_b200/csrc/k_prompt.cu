// k_prompt.cu -- causal attention over whole prompts: packed sequences of different
// lengths, grouped query heads, head dim 128, tcgen05, sm_100a.
//
//   o[t,h] = sum_{j <= t, same sequence} softmax_j(scale q[t,h] . k[j,g]) v[j,g],
//   g = h / (Hq / Hkv).
//
// The rows of a query tile are (token, query head of the group) pairs, so the heads of a
// group share every key and value tile and a short prompt still fills a tile.  A CTA takes
// 2 x 128 such rows (consecutive tokens) of one key/value head and walks their key blocks
// of 128 once, with one pass over the keys (running maximum and sum).  Per key block each
// half needs 2 x 2^21 multiply-adds (1024 tensor-core cycles for both) and 2^14
// exponentials (1024 cycles of the SM's 16 per clock): the two are equally scarce, so the
// halves alternate -- while one half's warps form exponentials, the tensor cores work for
// the other.  Warp roles, joined by bounded mbarrier waits:
//   * producer (one thread): the query rows once, then key and value blocks (32 KB each)
//     into one ring of five, in the order they are used;
//   * MMA (one thread): S = Q K^T of each half into its own tensor-memory tile, and
//     O += P V with P read from tensor memory (it lies over S: no shared memory is spent
//     on it, and S of the next block follows P V of this one in the pipe's order);
//   * two softmax warpgroups, one per half, one query row per thread: the row's 128
//     scores by one load, mask, maximum, exponentials, P in bf16 back to tensor memory,
//     32 keys at a time, so that P V of the first keys runs beside the exponentials of the
//     last (8192 tokens of 32 heads over 8: 467 us handed over whole, 426 in two parts, 422 in
//     four, 522 in eight; exponentials partly by a cubic on the FMA pipe gained nothing more).
// The reference maximum moves only when a block exceeds it by 2^8 (output and sum are then
// rescaled together): P stays below 256 and O / l is the same softmax.  Scores and sums are
// fp32; P is rounded to bf16, the type of the values it multiplies.
// The mask is applied before any maximum or exponential.  Value rows behind the end of the
// sequence (another sequence's) are zeroed in shared memory before use: 0 x NaN would reach
// the sum otherwise.
#include <cuda.h>

#include <mutex>

#include "seq_pages.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace stree {
namespace {

constexpr int kD = 128, kKB = 128, kM = 128;
constexpr int kThreads = 384;                  // four warps of loads and MMA, two softmax warpgroups
constexpr int kSlots = 5;
constexpr uint32_t kTile = 128 * 128 * 2, kHalf = kTile / 2;
constexpr float kLazyLog2 = 8.f;
constexpr uint32_t kSmem = 2 * kTile + kSlots * kTile + 1024;
constexpr int kParts = 4;                      // parts in which a block's P is handed over
constexpr int kMaxDevices = 64;

enum Bars { B_QF = 0, B_F = 1, B_E = B_F + kSlots, B_SF = B_E + kSlots, B_PF = B_SF + 2, B_OF = B_PF + 2 * kParts, B_DRAIN = B_OF + 2, kBars };

struct PromptArgs {
    const int32_t *cu;
    __nv_bfloat16 *o;
    int32_t *err;
    int total, batch, heads_q, heads_kv, group, tokens;   // tokens: of a half, 128 / group
    float scale_log2;
};

__global__ void __launch_bounds__(kThreads, 1)
prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PromptArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bars[kBars];
    __shared__ int tmp[33], found[2];
    __shared__ volatile int aborted;
    __shared__ uint32_t tmem_s;
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    const uint32_t q0 = ptx::smem_u32(smem), ring = q0 + 2 * kTile;
    const int tid = threadIdx.x, lane = tid & 31, warp = ptx::warp_index();

    pdl_start();
    if (blockIdx.x == gridDim.x - 1) {         // the error word
        PageCheck c{};
        c.cu = a.cu;
        c.batch = a.batch;
        c.total = a.total;
        check_pages(c, a.err);
        return;
    }
    const int g = blockIdx.x % a.heads_kv, span = 2 * a.tokens;
    auto tiles = [&](int b) {
        const int2 r = seq_range(a.cu, b, a.total);
        return (r.y - r.x + span - 1) / span;
    };
    block_find(a.batch, blockIdx.x / a.heads_kv, tiles, tmp, found);
    const int b = found[0];
    if (b < 0) return;                         // past the last tile
    const int2 seq = seq_range(a.cu, b, a.total);
    const int len = seq.y - seq.x;
    // A sequence's longest rows first: its last tile starts before its shorter ones.
    const int t0 = (tiles(b) - 1 - ((int)(blockIdx.x / a.heads_kv) - found[1])) * span;
    // Key blocks of each half (0: no token in it).
    int n_half[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int lo = t0 + i * a.tokens, hi = min(lo + a.tokens, len);
        n_half[i] = hi > lo ? (hi - 1) / kKB + 1 : 0;
    }
    const int n = max(n_half[0], n_half[1]);

    auto wait = [&](int i, uint32_t parity, int where) { return wait_one(&aborted, bar(i), parity, where); };
    auto warp_wait = [&](int i, uint32_t parity, int where) { return wait_warp(&aborted, bar(i), parity, where); };
    if (tid == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
        for (int i = 0; i < kBars; ++i) ptx::mbar_init(bar(i), i >= B_PF && i < B_OF ? 4 : 1);
        ptx::fence_mbar_init();
        aborted = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_s), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_s;              // S of both halves: 0, 128; O: 256, 384

    int loads = 0;
    if (warp < 4) {
        ptx::regs_less<56>();
        if (warp == 0) {
            if (ptx::elect_one()) {
                // -------------------------------------------------------- producer
                const uint32_t q_bytes = (uint32_t)(a.group * a.tokens) * 256u;
                const int halves = n_half[1] ? 2 : 1;
                ptx::mbar_expect_tx(bar(B_QF), q_bytes * halves);
                for (int i = 0; i < halves; ++i)
                    for (int hh = 0; hh < 2; ++hh)
                        ptx::tma_load_3d(q0 + i * kTile + hh * kHalf, &tm_q, hh * 64, g * a.group, seq.x + t0 + i * a.tokens, bar(B_QF));
#pragma unroll 1
                for (; loads < 2 * n; ++loads) {
                    const int s = loads % kSlots;
                    if (loads >= kSlots && !wait(B_E + s, (uint32_t)(loads / kSlots - 1), 1)) break;
                    ptx::mbar_expect_tx(bar(B_F + s), kTile);
                    const CUtensorMap *m = loads & 1 ? &tm_v : &tm_k;
                    for (int hh = 0; hh < 2; ++hh)
                        ptx::tma_load_3d(ring + s * kTile + hh * kHalf, m, hh * 64, g, seq.x + (loads >> 1) * kKB, bar(B_F + s));
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issue
            const uint32_t id_s = ptx::idesc_bf16_kk(kM, kKB), id_o = ptx::idesc_bf16_bmn(kM, kD);
            // Load number x (K of block i: 2 i, V: 2 i + 1) has arrived.
            auto arrived = [&](int x) { return warp_wait(B_F + x % kSlots, (uint32_t)(x / kSlots), 10); };
            auto scores = [&](int half, int i) {
                const uint64_t d_q = ptx::desc_kmajor_sw128(q0 + half * kTile),
                               d_k = ptx::desc_kmajor_sw128(ring + (2 * i % kSlots) * kTile);
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                    ptx::mma_f16(tmem + half * kKB, ptx::desc_at(d_q, (kk >> 2) * kHalf + (kk & 3) * 32),
                                 ptx::desc_at(d_k, (kk >> 2) * kHalf + (kk & 3) * 32), id_s, kk != 0);
                ptx::mma_commit(bar(B_SF + half));
            };
            // A part of a block's keys: P is handed over in parts.
            auto values = [&](int half, int i, int part) {
                const uint64_t d_v = ptx::desc_mnmajor_sw128(ring + ((2 * i + 1) % kSlots) * kTile, kHalf, 1024);
#pragma unroll
                for (int kk = part * (8 / kParts); kk < (part + 1) * (8 / kParts); ++kk)
                    ptx::mma_f16_ta(tmem + 256 + half * kD, tmem + half * kKB + kk * 8, ptx::desc_at(d_v, kk * 2048), id_o,
                                    (i | kk) != 0);
                if (part == kParts - 1 && i == n_half[half] - 1) ptx::mma_commit(bar(B_OF + half));
            };
            bool ok = warp_wait(B_QF, 0, 11) && arrived(0);
            if (ok && ptx::elect_one()) {
                ptx::tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (n_half[half]) scores(half, 0);
                if (kSlots < 2 * n) ptx::mma_commit(bar(B_E + 0));
            }
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                if (!(ok = arrived(2 * i + 1))) break;
                const int valid = len - i * kKB;
                if (valid < kKB) {             // the rows behind the sequence's end
                    uint8_t *v = smem + 2 * kTile + ((2 * i + 1) % kSlots) * kTile;
#pragma unroll 1
                    for (int e = lane; e < (kKB - valid) * 16; e += 32) {
                        const int r = valid + e / 16, c = e % 16;
                        *reinterpret_cast<uint4 *>(v + (c >> 3) * kHalf + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                }
                if (i + 1 < n && !(ok = arrived(2 * i + 2))) break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (i >= n_half[half] || !ok) continue;
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        if (!ok || !(ok = warp_wait(B_PF + kParts * half + part, (uint32_t)i, 12))) continue;
                        if (ptx::elect_one()) {
                            ptx::tc_fence_after();
                            values(half, i, part);
                            if (part == kParts - 1 && i + 1 < n_half[half]) scores(half, i + 1);
                        }
                        __syncwarp();
                    }
                }
                if (ok && ptx::elect_one()) {  // slots that another load will use
                    if (2 * i + 1 + kSlots < 2 * n) ptx::mma_commit(bar(B_E + (2 * i + 1) % kSlots));
                    if (2 * i + 2 + kSlots < 2 * n) ptx::mma_commit(bar(B_E + (2 * i + 2) % kSlots));
                }
                __syncwarp();
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax
        ptx::regs_more<224>();
        const int half = (warp >> 2) - 1, quad = warp & 3, nh = half ? n_half[1] : n_half[0];
        const int r = quad * 32 + lane;        // query row = tensor-memory lane
        const int token = t0 + half * a.tokens + r / a.group;
        const bool real = r < a.group * a.tokens && token < len;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t t_s = tmem + half * kKB + lanes, t_o = tmem + 256 + half * kD + lanes;
        // Blocks from here on reach past this half's first token.
        const int masked = (t0 + half * a.tokens + 1) / kKB;
        float m = -INFINITY, l = 0.f;
        bool run = true;
        for (int i = 0; i < nh; ++i) {
            if (!(run = warp_wait(B_SF + half, (uint32_t)i, 20))) break;
            ptx::tc_fence_after();
            uint32_t sv[kKB];
            ptx::tmem_ld128(t_s, sv);
            if (i >= masked) {
                const int lim = token - i * kKB;
#pragma unroll
                for (int key = 0; key < kKB; ++key)
                    if (key > lim) sv[key] = 0xff800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int key = 0; key < kKB; key += 2)
                mx[(key >> 1) & 3] = fmaxf(mx[(key >> 1) & 3], fmaxf(__uint_as_float(sv[key]), __uint_as_float(sv[key + 1])));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
            bool need = false;
            float f = 1.f;
            if (i == 0) {
                m = top;
            } else if (top > m + kLazyLog2) {
                need = true;
                f = ptx::ex2_approx(m - top);
                m = top;
            }
            // S of this block was issued after P V of the last one: O is complete.
            if (__any_sync(0xffffffffu, need)) {
                uint32_t ov[32];
#pragma unroll
                for (int c = 0; c < kD / 32; ++c) {
                    ptx::tmem_ld32(t_o + c * 32, ov);
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                    ptx::tmem_st32(t_o + c * 32, ov);
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), ref2 = make_float2(-ref, -ref);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < kParts; ++c) {
                constexpr int kPairs = kKB / 2 / kParts;
                uint32_t pk[kPairs];
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    const int key = 2 * (c * kPairs + e);
                    const float2 x = ptx::ffma2(make_float2(__uint_as_float(sv[key]), __uint_as_float(sv[key + 1])), scale2, ref2);
                    const float2 q = make_float2(ptx::ex2_approx(x.x), ptx::ex2_approx(x.y));
                    sum[e & 1] = ptx::fadd2(sum[e & 1], q);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(q.x, q.y);
                    pk[e] = *reinterpret_cast<const uint32_t *>(&h);
                }
                ptx::tmem_st16(t_s + c * kPairs, pk);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_PF + kParts * half + c));
            }
            l = l * f + ((sum[0].x + sum[1].x) + (sum[0].y + sum[1].y));
        }
        if (nh && run && warp_wait(B_OF + half, 0, 21)) {
            ptx::tc_fence_after();
            uint32_t ov[kD];
            ptx::tmem_ld128(t_o, ov);
            if (real) {
                const float inv = 1.f / l;     // the row's own token is never masked: l > 0
                __nv_bfloat16 *row = a.o + ((size_t)(seq.x + token) * a.heads_q + g * a.group + r % a.group) * kD;
#pragma unroll
                for (int c = 0; c < kD / 8; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(ov[8 * c + 2 * u]) * inv,
                                                                       __uint_as_float(ov[8 * c + 2 * u + 1]) * inv);
                        w[u] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    *reinterpret_cast<uint4 *>(row + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }

    // -------------------------------------------------------------------- teardown
    if (tid == 64 && aborted && a.err) latch_error(a.err, STREE_ERR_TIMEOUT, b, aborted, 0);
    if (warp == 1 && aborted && ptx::elect_one()) {
        ptx::mma_commit(bar(B_DRAIN));         // every issued MMA completes first
        ptx::mbar_wait(bar(B_DRAIN), 0);
    }
    if (warp == 0 && aborted) {
        ptx::mbar_wait(bar(B_QF), 0);
#pragma unroll 1
        for (int x = max(0, loads - kSlots); x < loads; ++x) ptx::mbar_wait(bar(B_F + x % kSlots), (uint32_t)((x / kSlots) & 1));
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

std::mutex g_mutex;
bool g_ready[kMaxDevices] = {};

cudaError_t prepare()
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_ready[dev]) {
        if ((e = cudaFuncSetAttribute(prompt_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem)) != cudaSuccess)
            return e;
        g_ready[dev] = true;
    }
    return cudaSuccess;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace stree

using namespace stree;

extern "C" stree_status stree_prompt_attention(const void *q, const void *k, const void *v, const int32_t *cu_seqlens,
                                               int total, int batch, int heads_q, int heads_kv, int head_dim,
                                               float scale, stree_dtype dtype, void *o, int32_t *err_out, void *stream)
{
    if (batch < 0 || total < 0 || heads_q < 1 || heads_kv < 1 || heads_q % heads_kv != 0 || heads_q / heads_kv > kM ||
        head_dim != kD || dtype != STREE_BF16)
        return STREE_ERR_UNSUPPORTED;
    if (!(scale > 0.f)) return STREE_ERR_INVALID_ARG;
    if (batch == 0) return STREE_OK;
    if (!cu_seqlens || (total > 0 && (!q || !k || !v || !o))) return STREE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(cu_seqlens, 4) || !aligned(err_out, 4))
        return STREE_ERR_MISALIGNED;
    PromptArgs a{};
    a.cu = cu_seqlens;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.err = err_out;
    a.total = total;
    a.batch = batch;
    a.heads_q = heads_q;
    a.heads_kv = heads_kv;
    a.group = heads_q / heads_kv;
    a.tokens = kM / a.group;
    a.scale_log2 = scale * 1.4426950408889634f;
    // Every sequence has at most one tile that it does not fill; no token, no tile.
    const long long tiles = total / (2 * a.tokens) + (batch < total ? batch : total);
    const long long grid = tiles * heads_kv + 1;
    if (grid > 0x7fffffffLL) return STREE_ERR_UNSUPPORTED;
    if (prepare() != cudaSuccess) return STREE_ERR_CUDA;
    CUtensorMap m_q{}, m_k{}, m_v{};
    if (total > 0 && (!encode_heads(&m_q, q, total, heads_q, a.group, a.tokens) ||
                      !encode_heads(&m_k, k, total, heads_kv, 1, kKB) || !encode_heads(&m_v, v, total, heads_kv, 1, kKB)))
        return STREE_ERR_CUDA;
    return launch_pdl(prompt_attention_kernel, dim3((unsigned)grid), kThreads, kSmem, static_cast<cudaStream_t>(stream), m_q,
                      m_k, m_v, a) == cudaSuccess
               ? STREE_OK
               : STREE_ERR_CUDA;
}
