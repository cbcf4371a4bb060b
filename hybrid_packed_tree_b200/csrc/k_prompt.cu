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
// the other.
//
// The grid holds a CTA per tile (an upper bound: each sequence has at most one that it does not
// fill), a sequence's longest tiles first.  A CTA that is done takes over one that was not
// launched yet (cluster launch control) and loads its keys while its last rows are still written:
// per tile, setting up anew cost 7.6 us.  64 sequences of 16 to 1024 tokens, 32 heads over 8: 86 us
// with a CTA launched for each tile, 79 so; 8192 tokens: 423 and 419; small calls pay
// 0.4 to 1.2 us for it (97 tokens: 9.2 and 9.5; 14 x 64 tokens: 10.6 and 11.7).  The next tile is taken when all roles have begun
// the last one; taken one earlier, the packed batch took 87 us (the tiles are shared out before
// it shows who is done first).  Warp roles, joined by bounded mbarrier waits:
//   * scheduler (one warp): the next tile, found among the sequences;
//   * producer (one thread): a tile's query rows, then key and value blocks (32 KB each)
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
// Times above are of one call in loops too short for the card's power cap; under it, among calls on changing
// inputs, 8192 tokens take 485 us and a packed batch of 5604 tokens 70 us.  The stores below were compared so.
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

enum Bars {
    B_QF = 0, B_QE, B_F, B_E = B_F + kSlots, B_SF = B_E + kSlots, B_PF = B_SF + 2, B_OF = B_PF + 2 * kParts, B_OE = B_OF + 2,
    B_TF = B_OE + 2, B_TE = B_TF + 2, B_NEXT = B_TE + 2, B_DRAIN, kBars
};
constexpr int kTileReaders = 1 + 1 + 8;        // producer, MMA warp, softmax warps

struct PromptArgs {
    const int32_t *cu;
    __nv_bfloat16 *o;
    int32_t *err;
    int total, batch, heads_q, heads_kv, group, tokens;   // tokens: of a half, 128 / group
    uint32_t wait_ns;                          // limit of a wait
    int fault;                                 // test hook: 1 withholds the first part of P of a CTA's first tile
    float scale_log2;
};

// A tile of 2 x `tokens` tokens of one sequence and key/value head, as the scheduler hands it out.
struct Tile {
    int row, len, t0, g;                       // the sequence's first row and length, the tile's first token, head
    int n[2];                                  // key blocks of each half (0: no token in it)
    int more, pad;                             // 0: there is no tile
};

// The error word, by one warp.
__device__ __forceinline__ void check_offsets(const PromptArgs &a, int lane)
{
    if (!a.err) return;
    if (lane < 4) a.err[lane] = 0;
    __syncwarp();
    for (int b = lane; b < a.batch; b += 32) {
        const int lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1);
        if (lo < 0 || hi < lo || hi > a.total) latch_error(a.err, STREE_ERR_BAD_SEQ, b, lo, hi);
    }
}

// Tile number x of the list (a sequence's tiles from its last, the longest, to its first), by one
// warp, four sequences a lane; false past the list's end.  `b0` and `base`: a group of sequences
// and the tiles before it, from which the search goes on when x lies behind them.
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int x, int lane, int &b0, int &base, Tile &t)
{
    const int span = 2 * a.tokens;
    if (x < base) b0 = base = 0;
    for (; b0 < a.batch; b0 += 128) {
        int2 r[4];
        int count[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int b = b0 + 4 * lane + e;
            r[e] = b < a.batch ? seq_range(a.cu, b, a.total) : make_int2(0, 0);
            count[e] = (r[e].y - r[e].x + span - 1) / span;
            sum += count[e];
        }
        int upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += u;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, x < base + upto);
        if (here) {
            int at = x - (base + upto - sum), row = 0, len = 0, tiles = 0;   // of use in the lane that holds x
            bool found = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!found && at < count[e]) {
                    row = r[e].x;
                    len = r[e].y - r[e].x;
                    tiles = count[e];
                    found = true;
                }
                if (!found) at -= count[e];
            }
            const int w = __ffs(here) - 1;
            t.row = __shfl_sync(0xffffffffu, row, w);
            t.len = __shfl_sync(0xffffffffu, len, w);
            t.t0 = __shfl_sync(0xffffffffu, tiles - 1 - at, w) * span;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int lo = t.t0 + i * a.tokens, hi = min(lo + a.tokens, t.len);
                t.n[i] = hi > lo ? (hi - 1) / kKB + 1 : 0;
            }
            return true;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

__global__ void __launch_bounds__(kThreads, 1)
prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PromptArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bars[kBars];
    __shared__ alignas(16) uint4 answer;
    __shared__ alignas(16) Tile tiles_s[2];
    __shared__ volatile int aborted;
    __shared__ uint32_t tmem_s;
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    const uint32_t q0 = ptx::smem_u32(smem), ring = q0 + 2 * kTile;
    const int tid = threadIdx.x, lane = tid & 31, warp = ptx::warp_index();

    auto wait = [&](int i, uint32_t parity, int where) { return wait_one(&aborted, bar(i), parity, where, a.wait_ns); };
    auto warp_wait = [&](int i, uint32_t parity, int where) { return wait_warp(&aborted, bar(i), parity, where, a.wait_ns); };
    if (tid == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
        for (int i = 0; i < kBars; ++i)
            ptx::mbar_init(bar(i), (i >= B_PF && i < B_OF) || i == B_OE || i == B_OE + 1 ? 4 : i == B_TE || i == B_TE + 1 ? kTileReaders : 1);
        ptx::fence_mbar_init();
        aborted = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_s), 512);
        ptx::tmem_relinquish();
    }
    pdl_start();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_s;              // S of both halves: 0, 128; O: 256, 384
    // Tile number k of this CTA (the last one has more = 0), read from its slot.
    auto tile_at = [&](int k) {
        const int4 *src = reinterpret_cast<const int4 *>(&tiles_s[k & 1]);
        const int4 x = src[0], y = src[1];
        Tile t;
        t.row = x.x;
        t.len = x.y;
        t.t0 = x.z;
        t.g = x.w;
        t.n[0] = y.x;
        t.n[1] = y.y;
        t.more = y.z;
        return t;
    };

    int loads = 0, requests = 0, q_loads = 0;
    bool pending = false;                      // a request of the scheduler whose answer has not been read
    if (warp == 0) {
        if (ptx::elect_one()) {
            // ------------------------------------------------------------ producer
            const uint32_t q_bytes = (uint32_t)(a.group * a.tokens) * 256u;
            bool ok = true;
#pragma unroll 1
            for (int k = 0; ok; ++k) {
                if (!wait(B_TF + (k & 1), (uint32_t)(k >> 1), 1)) break;
                const Tile t = tile_at(k);
                ptx::mbar_arrive(bar(B_TE + (k & 1)));
                if (!t.more) break;
                if (k > 0 && !wait(B_QE, (uint32_t)(k - 1), 2)) break;
                const int halves = t.n[1] ? 2 : 1, n = max(t.n[0], t.n[1]);
                ptx::mbar_expect_tx(bar(B_QF), q_bytes * halves);
                ++q_loads;
                for (int i = 0; i < halves; ++i)
                    for (int hh = 0; hh < 2; ++hh)
                        ptx::tma_load_3d(q0 + i * kTile + hh * kHalf, &tm_q, hh * 64, t.g * a.group, t.row + t.t0 + i * a.tokens, bar(B_QF));
#pragma unroll 1
                for (int x = 0; x < 2 * n; ++x, ++loads) {
                    const int s = loads % kSlots;
                    if (loads >= kSlots && !(ok = wait(B_E + s, (uint32_t)(loads / kSlots - 1), 3))) break;
                    ptx::mbar_expect_tx(bar(B_F + s), kTile);
                    const CUtensorMap *m = x & 1 ? &tm_v : &tm_k;
                    for (int hh = 0; hh < 2; ++hh)
                        ptx::tma_load_3d(ring + s * kTile + hh * kHalf, m, hh * 64, t.g, t.row + (x >> 1) * kKB, bar(B_F + s));
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issue
        const uint32_t id_s = ptx::idesc_bf16_kk(kM, kKB), id_o = ptx::idesc_bf16_bmn(kM, kD);
        int x0 = 0, done[2] = {0, 0}, uses[2] = {0, 0};   // loads, key blocks and tiles (of each half) before this tile
        bool ok = true;
#pragma unroll 1
        for (int k = 0; ok; ++k) {
            if (!(ok = warp_wait(B_TF + (k & 1), (uint32_t)(k >> 1), 9))) break;
            const Tile t = tile_at(k);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_TE + (k & 1)));
            if (!t.more) break;
            const int n = max(t.n[0], t.n[1]);
            // Load number x of the tile (K of block i: 2 i, V: 2 i + 1): its slot, and its arrival.
            auto slot = [&](int x) { return (x0 + x) % kSlots; };
            auto arrived = [&](int x) { return warp_wait(B_F + slot(x), (uint32_t)((x0 + x) / kSlots), 10); };
            auto scores = [&](int half, int i) {
                const uint64_t d_q = ptx::desc_kmajor_sw128(q0 + half * kTile), d_k = ptx::desc_kmajor_sw128(ring + slot(2 * i) * kTile);
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                    ptx::mma_f16(tmem + half * kKB, ptx::desc_at(d_q, (kk >> 2) * kHalf + (kk & 3) * 32),
                                 ptx::desc_at(d_k, (kk >> 2) * kHalf + (kk & 3) * 32), id_s, kk != 0);
                ptx::mma_commit(bar(B_SF + half));
            };
            // A part of a block's keys: P is handed over in parts.
            auto values = [&](int half, int i, int part) {
                const uint64_t d_v = ptx::desc_mnmajor_sw128(ring + slot(2 * i + 1) * kTile, kHalf, 1024);
#pragma unroll
                for (int kk = part * (8 / kParts); kk < (part + 1) * (8 / kParts); ++kk)
                    ptx::mma_f16_ta(tmem + 256 + half * kD, tmem + half * kKB + kk * 8, ptx::desc_at(d_v, kk * 2048), id_o,
                                    (i | kk) != 0);
                if (part == kParts - 1 && i == t.n[half] - 1) ptx::mma_commit(bar(B_OF + half));
            };
            if (!(ok = warp_wait(B_QF, (uint32_t)k, 11) && arrived(0))) break;
            if (ptx::elect_one()) {
                ptx::tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (t.n[half]) scores(half, 0);
                ptx::mma_commit(bar(B_E + slot(0)));
                if (n == 1) ptx::mma_commit(bar(B_QE));
            }
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                if (!(ok = arrived(2 * i + 1))) break;
                const int valid = t.len - i * kKB;
                if (valid < kKB) {             // the rows behind the sequence's end
                    uint8_t *v = smem + 2 * kTile + slot(2 * i + 1) * kTile;
#pragma unroll 1
                    for (int e = lane; e < (kKB - valid) * 16; e += 32) {
                        const int r = valid + e / 16, c = e % 16;
                        *reinterpret_cast<uint4 *>(v + (c >> 3) * kHalf + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
                if (i + 1 < n && !(ok = arrived(2 * i + 2))) break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (i >= t.n[half] || !ok) continue;
                    // The last tile's output of this half has been read before this one's begins.
                    if (i == 0 && uses[half] > 0 && !(ok = warp_wait(B_OE + half, (uint32_t)(uses[half] - 1), 14))) continue;
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        if (!ok || !(ok = warp_wait(B_PF + kParts * half + part, (uint32_t)(done[half] + i), 12))) continue;
                        if (ptx::elect_one()) {
                            ptx::tc_fence_after();
                            values(half, i, part);
                            if (part == kParts - 1 && i + 1 < t.n[half]) scores(half, i + 1);
                        }
                        __syncwarp();
                    }
                }
                if (ok && ptx::elect_one()) {  // the slots of this block's V and of the next one's K; Q after the last K
                    ptx::mma_commit(bar(B_E + slot(2 * i + 1)));
                    if (i + 1 < n) ptx::mma_commit(bar(B_E + slot(2 * i + 2)));
                    if (i + 2 == n) ptx::mma_commit(bar(B_QE));
                }
                __syncwarp();
            }
            x0 += 2 * n;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                done[half] += t.n[half];
                uses[half] += t.n[half] ? 1 : 0;
            }
        }
        // No commit may arrive in the shared memory of a CTA that has ended, and no MMA run on.
        if (ptx::elect_one()) {
            ptx::mma_commit(bar(B_DRAIN));
            ptx::mbar_wait(bar(B_DRAIN), 0);
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- scheduler
        // Tiles are taken from the grid's list as CTAs that were not launched yet, one ahead of the work.
        // Block 0's place in it is the error word, so that this is cleared before the rest.
        int x = blockIdx.x, b0 = 0, base = 0;
        bool ok = true;
#pragma unroll 1
        for (int k = 0; ok;) {
            Tile t{};
            bool some = false;
            if (x == 0) check_offsets(a, lane);
            else if (x > 0 && (some = find_tile(a, (x - 1) / a.heads_kv, lane, b0, base, t))) t.g = (x - 1) % a.heads_kv;
            t.more = some ? 1 : 0;
            if (some || x < 0) {
                if (lane == 0) {
                    int4 *dst = reinterpret_cast<int4 *>(&tiles_s[k & 1]);
                    dst[0] = make_int4(t.row, t.len, t.t0, t.g);
                    dst[1] = make_int4(t.n[0], t.n[1], t.more, 0);
                    ptx::mbar_arrive(bar(B_TF + (k & 1)));
                }
                __syncwarp();
                if (x < 0) break;
                // The next one is taken when every role has begun this one: taken earlier, the tiles would be
                // shared out before it is known which CTAs are done first.
                if (!(ok = warp_wait(B_TE + (k & 1), (uint32_t)(k >> 1), 30))) break;
                ++k;
            }
            if (lane == 0) {
                ptx::fence_proxy_async_smem(); // the last answer has been read
                ptx::mbar_expect_tx(bar(B_NEXT), 16);
                ptx::clc_request(ptx::smem_u32(&answer), bar(B_NEXT));
            }
            __syncwarp();
            pending = true;
            if (!(ok = warp_wait(B_NEXT, (uint32_t)requests, 31))) break;
            pending = false;
            ++requests;
            x = ptx::clc_answer(ptx::smem_u32(&answer));
            __syncwarp();
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- softmax
        const int half = (warp >> 2) - 1, quad = warp & 3;
        const int r = quad * 32 + lane;        // query row = tensor-memory lane
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t t_s = tmem + half * kKB + lanes, t_o = tmem + 256 + half * kD + lanes;
        const bool wide = (reinterpret_cast<uintptr_t>(a.o) & 31) == 0;   // 32-byte stores
        int done = 0, uses = 0;                // key blocks and tiles of this half before this tile
        bool run = true;
#pragma unroll 1
        for (int k = 0; run; ++k) {
            if (!(run = warp_wait(B_TF + (k & 1), (uint32_t)(k >> 1), 19))) break;
            const Tile t = tile_at(k);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_TE + (k & 1)));
            if (!t.more) break;
            const int nh = half ? t.n[1] : t.n[0];
            if (nh == 0) continue;
            const int token = t.t0 + half * a.tokens + r / a.group;
            // Blocks from here on reach past this half's first token.
            const int masked = (t.t0 + half * a.tokens + 1) / kKB;
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int i = 0; i < nh; ++i) {
                if (!(run = warp_wait(B_SF + half, (uint32_t)(done + i), 20))) break;
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
                    if (lane == 0 && !(c == 0 && a.fault && k + i == 0)) ptx::mbar_arrive(bar(B_PF + kParts * half + c));
                }
                l = l * f + ((sum[0].x + sum[1].x) + (sum[0].y + sum[1].y));
            }
            if (!run || !(run = warp_wait(B_OF + half, (uint32_t)uses, 21))) break;
            ptx::tc_fence_after();
            uint32_t ov[kD];
            ptx::tmem_ld128(t_o, ov);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_OE + half));
            if (r < a.group * a.tokens && token < t.len) {
                const float inv = 1.f / l;     // the row's own token is never masked: l > 0
                __nv_bfloat16 *row = a.o + ((size_t)(t.row + token) * a.heads_q + t.g * a.group + r % a.group) * kD;
#pragma unroll
                for (int c = 0; c < kD / 16; ++c) {
                    uint32_t w[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(ov[16 * c + 2 * u]) * inv,
                                                                       __uint_as_float(ov[16 * c + 2 * u + 1]) * inv);
                        w[u] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    if (wide) {                // half the accesses: 490 -> 482 us on 8192 tokens, 73 -> 69 packed
                        ptx::st_global_32b(row + 16 * c, w);
                    } else {
                        *reinterpret_cast<uint4 *>(row + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4 *>(row + 16 * c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
            }
            done += nh;
            ++uses;
        }
    }

    // -------------------------------------------------------------------- teardown
    ptx::tc_fence_before();
    __syncthreads();                           // all roles have ended: `aborted` no longer changes
    if (aborted) {
        if (tid == 0 && a.err) latch_error(a.err, STREE_ERR_TIMEOUT, -1, aborted, 0);
        // What may still land in shared memory: copies, and an answer that was not waited for.
        if (q_loads > 0) {                     // the producer's lane
            ptx::mbar_wait(bar(B_QF), (uint32_t)((q_loads - 1) & 1));
#pragma unroll 1
            for (int x = max(0, loads - kSlots); x < loads; ++x) ptx::mbar_wait(bar(B_F + x % kSlots), (uint32_t)((x / kSlots) & 1));
        }
        if (pending) ptx::mbar_wait(bar(B_NEXT), (uint32_t)(requests & 1));
        __syncthreads();
    }
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
    const WaitHook hook = wait_hook();
    a.wait_ns = hook.limit_ns;
    a.fault = hook.fault;
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
