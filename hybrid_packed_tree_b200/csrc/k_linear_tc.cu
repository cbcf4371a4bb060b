// k_linear_tc.cu -- linear attention with a decay for each head over whole prompts, in
// chunks of 128 tokens on the tensor cores (bf16, dk = 128, dv = 128 or 64), sm_100a.
//
// With L_t the sum of log2 alpha over the chunk up to token t, C its last token and S the
// state before the chunk:
//   P_ij = 2^(L_i - L_j) beta_j (q_i . k_j) for j <= i (+ skip where j = i), 0 beyond
//   O    = P V + diag(2^L) Q S^T
//   S'   = 2^L_C S + sum_j (w_j v_j) k_j^T,  w_j = 2^(L_C - L_j) beta_j
// the state's with three operands for one (below): six 128 x 128 x 128 products a chunk.  No
// exponent above is positive for alpha <= 1.
//
// A CTA walks the chunks of one sequence and 128 value columns (one head of 128, or two of 64 that
// share keys and queries: their Q K^T is one product).  Few sequences of many tokens are
// cut into segments.  Three launches: the states and log decays of the middle segments from a zero
// state, left in the workspace; beside them, on other SMs, the whole walk of the first, a shorter
// one; and the walks of the others, each from the first one's state folded with those between (the
// recurrence is linear).
//
// Precision.  P and the copy of S that Q multiplies are rounded to bf16 (they only enter o,
// itself bf16).  The state is kept in fp32 registers and receives w_j v_j as three bf16 parts
// (24 bits), so its products are those of fp32.  L is summed in 64 bits and differences of it are taken
// before they are rounded to floats: over a block of 32 tokens, to a chunk's end, and between blocks.  The
// exponents of P and of Q S^T's scale are the sum or difference of two such floats, each off by at most 2^-24 of
// itself: 2^-11 together where a block has 31 zero decays, 2^-15 with one or two, and P is rounded to bf16 (2^-9).
//
// Warp roles (16 warps, bounded mbarrier waits): a producer (TMA: Q, V, K tiles of 32 KB into a
// ring of five), two MMA issuers (of P and O, and of the state's update, so that neither waits for
// the other's operands), a gate warp (L, w and the factors of P; two of them in the state-only launch),
// four warps for P and O (a token per thread; O leaves by one tensor copy a warp), and eight
// for the state (a row of S per thread and half of its columns; they also scale Q S^T, a token
// and half of the columns): they read V by columns and put the three parts of w v into tensor
// memory as the A operand, 16 tokens at a time in two alternating buffers for each half, then add the product
// to their registers and write the bf16 copy of S for the next chunk's Q S^T.
//
// 8192 tokens of 32 heads of 128 x 128 (205 MB): 91 us in a loop of one call, 102 among calls on changing
// inputs (4802 by the walk on the CUDA cores); twelve
// packed sequences of 4956 tokens in all, 80 heads of 64 x 128: 84 us either way.  A chunk takes 5750
// cycles, against 3100 of the tensor cores and 3800 of shared memory (operands, copies, rows of O):
// the loop that bounds it runs over the warps of P and O (O's rows read and sent out 1500, P 2000 for
// the first tokens and 2800 for the last, P V 800, Q K^T of the next chunk between).
//
// P below the diagonal 32 x 32 blocks is a product of a row factor 2^(L_i - L_J) and a column
// factor 2^(L_J - L_j) beta_j, J the last token of j's block: both at most 1, and one exponential per
// row and block instead of one per pair.
#include <cuda.h>

#include <mutex>

#include "linear.cuh"
#include "seq_pages.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace stree {
namespace {

constexpr int kC = 128;                        // tokens per chunk; also dk and the value columns of a CTA
constexpr int kThreads = 512;
// Tiles of the load ring: the state-only launch has the room of S's copy and of O's rows for one more.
__host__ __device__ constexpr int ring_slots(bool state) { return state ? 6 : 5; }
constexpr int kMaxSlots = 6;
constexpr uint32_t kTile = 128 * 128 * 2, kHalf = kTile / 2;
// log2 of a decay of zero.  The least float is 2^-149, so that 2^kLogZero is zero however it is formed; and no further
// down, since sums of it within a chunk are rounded to floats.  (2^-130, as exp2f gives it, left 7e-40 of a state.)
constexpr float kLogZero = -160.f;
constexpr int kMaxSegments = 9;
// Length of the first segment to the others': a chunk of the whole walk takes 4.3 us, of the state alone 2.4.
constexpr int kFirstWeight = 9, kOtherWeight = 16;
constexpr int kMaxDevices = 64;

enum Bars {
    B_F = 0, B_E = B_F + kMaxSlots, B_GF = B_E + kMaxSlots, B_GE = B_GF + 2, B_SF = B_GE + 2, B_PF, B_OQ, B_OF, B_OE, B_SOP,
    B_WF, B_WE = B_WF + 4, B_DF = B_WE + 4, B_DRAIN = B_DF + 2, kBars = B_DRAIN + 2
};

// Tensor memory: Q K^T, then P over it (of every 32 columns, 16 for a head); O; the state's
// update; the parts of w v.
constexpr uint32_t kColP = 0, kColO = 128, kColD = 256, kColW = 384;

// The state-only launch has no P and no O: their columns hold two more of the parts' buffers and a
// second one for the update.
__device__ __forceinline__ uint32_t state_col_w(int s) { return s < 2 ? kColP + s * 64 : kColW + (s - 2) * 64; }
__device__ __forceinline__ uint32_t state_col_d(int i) { return i & 1 ? kColO : kColD; }

struct Gates {                                 // of one chunk, per head
    float rel[2][kC];                          // L_i less L at the end of the block before i's
    float beta[2][kC];
    float fac[2][kC];                          // 2^(L at the end of j's block - L_j) beta_j
    float w[2][kC];
    float step[2][4][4];                       // of block i: log decay from the end of block J < i to its start, and [3] from the chunk's
    double all[2];                             // of the whole chunk
};

struct TcArgs {
    const float *alpha, *beta, *skip, *S0;
    const int32_t *cu;
    __nv_bfloat16 *o;
    float *S_new;
    float *seg_state;                          // [item][segments - 1][128][128]: of every segment but the last
    double *seg_log;                           // [item][segments - 1][even, odd chunks][2]: the first's is not used
    int32_t *err;
    int total, batch, heads_v, heads_k, per_seq, segments;   // per_seq: 128-column items of a sequence
    int seg_first, seg_count;                  // of this launch
    uint32_t wait_ns;                          // limit of a wait
    int fault;                                 // test hook: 1 withholds the first hand-over of a CTA's first chunk
};

constexpr uint32_t kStage = 4 * 4096;          // rows of O on their way out: 32 rows of 64 columns a warp
constexpr uint32_t kSmem = 6 * kTile + kStage + 2 * sizeof(Gates) + 1024;

// Rows [valid, 128) of a tile of tokens become zero (they belong to another sequence).
__device__ __forceinline__ void zero_rows(uint8_t *tile, int valid, int lane)
{
#pragma unroll 1
    for (int e = lane; e < (kC - valid) * 16; e += 32) {
        const int r = valid + e / 16, c = e % 16;
        *reinterpret_cast<uint4 *>(tile + (c >> 3) * kHalf + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// NH: heads in the CTA's 128 value columns.  kState: the first launch of a split (state only).
template <int NH, bool kState>
__global__ void __launch_bounds__(kThreads, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const TcArgs a)
{
    constexpr int kDv = kC / NH;
    constexpr int kLoads = kState ? 2 : 3;     // tiles per chunk: K, (Q,) V
    constexpr int kSlots = ring_slots(kState);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bars[kBars];
    __shared__ volatile int aborted;
    __shared__ uint32_t tmem_s;
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sop = smem + 5 * kTile;           // the bf16 state, K-major
    uint8_t *stage = smem + 6 * kTile;
    Gates *gates = reinterpret_cast<Gates *>(stage + kStage);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    const uint32_t ring = ptx::smem_u32(smem), sop_u = ptx::smem_u32(sop);
    const int tid = threadIdx.x, lane = tid & 31, warp = ptx::warp_index();

    // The first segment's launch runs beside the state-only one, which lets it start once the kernels
    // before are done, and waits for that one's end at its own.
    const bool beside = !kState && a.segments > 1 && a.seg_first == 0;
    if (!beside) wait_dependency();
    launch_dependents();
    // The error word, by the first block of a call's first launch: cleared before any wait of the call can run
    // out.  (By the last block it was cleared when the first CTAs had ended, with what they had reported.)
    const bool first = kState || (a.seg_first == 0 && a.segments == 1);
    if (first && blockIdx.x == 0) {
        PageCheck c{};
        c.cu = a.cu;
        c.batch = a.batch;
        c.total = a.total;
        check_pages(c, a.err);
        return;
    }
    const int nth = blockIdx.x - (first ? 1 : 0);
    const int seg = a.seg_first + nth % a.seg_count, flat = nth / a.seg_count;   // flat: (sequence, 128-column item)
    const int item = flat % a.per_seq, b = flat / a.per_seq;
    const int head0 = item * NH, g = head0 / (a.heads_v / a.heads_k);
    const int2 seq = seq_range(a.cu, b, a.total);
    const int len = seq.y - seq.x, chunks = (len + kC - 1) / kC;
    const auto begin = [&](int s) {
        return s == 0 ? 0 : (int)((long long)chunks * (kFirstWeight + kOtherWeight * (s - 1)) / (kFirstWeight + kOtherWeight * (a.segments - 1)));
    };
    const int c0 = begin(seg), n = begin(seg + 1) - c0;
    const bool last = seg == a.segments - 1;
    if (n == 0 && !kState && seg > 0 && !last) return;   // nothing to put out

    auto wait = [&](int i, uint32_t parity, int where) { return wait_one(&aborted, bar(i), parity, where, a.wait_ns); };
    auto warp_wait = [&](int i, uint32_t parity, int where) { return wait_warp(&aborted, bar(i), parity, where, a.wait_ns); };
    auto both_wait = [&](int i, uint32_t i_parity, int j, uint32_t j_parity, int where) {
        const bool ok = wait(i, i_parity, where) && wait(j, j_parity, where + 1);
        return __all_sync(0xffffffffu, ok) != 0;
    };
    if (tid == 0) {
        ptx::prefetch_tensormap(&tm_q);
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
        for (int i = 0; i < kBars; ++i) {
            const int count = i == B_OE || (i >= B_WF && i < B_WE)   ? 4
                              : i == B_SOP                           ? 8
                              : i >= B_E && i < B_E + kMaxSlots && !kState ? 2
                              : i == B_PF || i == B_GE || i == B_GE + 1 ? 12
                                                                     : 1;
            ptx::mbar_init(bar(i), count);
        }
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
    const uint32_t tmem = tmem_s;
    // Load numbers of a chunk: Q, V, K.  In this order a load takes the slot of V or K of the chunk
    // before last, or of Q of the last one, which is free first; with K first, V waited for the
    // last chunk's update and came late.
    auto load_q = [&](int i) { return kLoads * i; };
    auto load_v = [&](int i) { return kLoads * i + kLoads - 2; };
    auto load_k = [&](int i) { return kLoads * i + kLoads - 1; };

    // Tokens t0 .. t0 + 15 of chunk i as w v, for the value columns of this warp's quarter of the lanes, in
    // three parts of 8 columns, `stride` apart, from `col` on.
    auto form = [&](int i, int t0, uint32_t col, uint32_t stride) {
        const Gates &G = gates[i & 1];
        const int x = load_v(i), valid = min(kC, len - (c0 + i) * kC), quad = warp & 3;
        const int h = NH == 2 ? quad >> 1 : 0;
        // This lane's row address for ldmatrix: token lane % 8 of eight, the warp's columns 8 (lane / 8) ..
        const uint32_t v = ring + (x % kSlots) * kTile + (quad >> 1) * kHalf + (lane & 7) * 128 +
                           ((((quad & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
        const uint32_t t_w = tmem + col + ((uint32_t)(quad * 32) << 16);
        // Transposed 8 x 8 tiles: a register is two tokens (2 (lane % 4), + 1) of column lane / 4.
        const int t = t0 + (lane & 3) * 2;
        uint32_t raw[2][4];
        ldsm4_t(v + t0 * 128, raw[0]);
        ldsm4_t(v + t0 * 128 + 1024, raw[1]);
        const float2 w[2] = {*reinterpret_cast<const float2 *>(&G.w[h][t]), *reinterpret_cast<const float2 *>(&G.w[h][t + 8])};
        float2 y[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c = 0; c < 4; ++c) y[e][c] = ptx::fmul2(w[e], make_float2(low(raw[e][c]), high(raw[e][c])));
        if (t0 + 16 > valid)       // another sequence's rows
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    y[e][c].x = t + 8 * e < valid ? y[e][c].x : 0.f;
                    y[e][c].y = t + 8 * e + 1 < valid ? y[e][c].y : 0.f;
                }
        // Three parts of eight bits each, cut off rather than rounded: their sum is exact.
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            uint32_t p[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t bx = __float_as_uint(y[e][c].x), by = __float_as_uint(y[e][c].y);
                    p[e][c] = __byte_perm(bx, by, 0x7632);
                    if (part < 2)
                        y[e][c] = ptx::ffma2(make_float2(low(p[e][c]), high(p[e][c])), make_float2(-1.f, -1.f), y[e][c]);
                }
            ptx::tmem_st16x8(t_w + part * stride, p[0][0], p[0][1], p[1][0], p[1][1]);
            ptx::tmem_st16x8(t_w + (16u << 16) + part * stride, p[0][2], p[0][3], p[1][2], p[1][3]);
        }
    };
    // The parts are there: to be followed by one arrival a warp.
    auto formed = [&] {
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
    };

    auto arrived = [&](int x, int where) { return warp_wait(B_F + x % kSlots, (uint32_t)(x / kSlots), where); };
    auto slot = [&](int x) { return ring + (x % kSlots) * kTile; };
    auto release = [&](int x) {                // a slot that another load will use
        if (x + kSlots < kLoads * n) ptx::mma_commit(bar(B_E + x % kSlots));
    };

    int loads = 0;
    if (warp < 4) {
        if (warp == 0) {
            if (ptx::elect_one()) {
                // ------------------------------------------------------------ producer
#pragma unroll 1
                for (; loads < kLoads * n; ++loads) {
                    const int s = loads % kSlots, i = loads / kLoads, what = loads % kLoads;
                    if (loads >= kSlots && !wait(B_E + s, (uint32_t)(loads / kSlots - 1), 1)) break;
                    const bool is_v = what == kLoads - 2;
                    const CUtensorMap *m = is_v ? &tm_v : what == kLoads - 1 ? &tm_k : &tm_q;
                    ptx::mbar_expect_tx(bar(B_F + s), kTile);
                    for (int hh = 0; hh < 2; ++hh)
                        ptx::tma_load_3d(ring + s * kTile + hh * kHalf, m, hh * 64, is_v ? item : g, seq.x + (c0 + i) * kC, bar(B_F + s));
                }
            }
        } else if (warp == 1 && !kState) {
            // ------------------------------------------------------------ MMA issue: P and O
            const uint32_t id_kk = ptx::idesc_bf16_kk(kC, kC), id_pv = ptx::idesc_bf16_bmn(kC, kDv);
            const uint64_t d_s = ptx::desc_kmajor_sw128(sop_u);
            bool ok = true;
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const int valid = min(kC, len - (c0 + i) * kC);
                // The descriptors of a tile's steps are made from one per tile.
                const uint64_t d_q = ptx::desc_kmajor_sw128(slot(load_q(i))), d_k = ptx::desc_kmajor_sw128(slot(load_k(i))),
                               d_v = ptx::desc_mnmajor_sw128(slot(load_v(i)), kHalf, 1024);
                if (!(ok = arrived(load_q(i), 11) && arrived(load_k(i), 10))) break;
                if (ptx::elect_one()) {
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kC / 16; ++kk)
                        ptx::mma_f16(tmem + kColP, ptx::desc_at(d_q, (kk >> 2) * kHalf + (kk & 3) * 32),
                                     ptx::desc_at(d_k, (kk >> 2) * kHalf + (kk & 3) * 32), id_kk, kk != 0);
                    ptx::mma_commit(bar(B_SF));
                    release(load_k(i));
                }
                __syncwarp();
                // Q S^T, when the last chunk's O has been read.
                if (!(ok = warp_wait(B_SOP, (uint32_t)i, 12)) || (i > 0 && !(ok = warp_wait(B_OE, (uint32_t)(i - 1), 13)))) break;
                if (ptx::elect_one()) {
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kC / 16; ++kk)
                        ptx::mma_f16(tmem + kColO, ptx::desc_at(d_q, (kk >> 2) * kHalf + (kk & 3) * 32),
                                     ptx::desc_at(d_s, (kk >> 2) * kHalf + (kk & 3) * 32), id_kk, kk != 0);
                    ptx::mma_commit(bar(B_OQ));
                    release(load_q(i));
                    release(load_q(i));        // no other reader
                }
                __syncwarp();
                if (!(ok = arrived(load_v(i), 15))) break;
                if (valid < kC) zero_rows(smem + (load_v(i) % kSlots) * kTile, valid, lane);
                if (!(ok = warp_wait(B_PF, (uint32_t)i, 16))) break;
                if (ptx::elect_one()) {
                    ptx::tc_fence_after();
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh)
#pragma unroll
                        for (int kk = 0; kk < kC / 16; ++kk)
                            ptx::mma_f16_ta(tmem + kColO + hh * kDv, tmem + kColP + (kk >> 1) * 32 + hh * 16 + (kk & 1) * 8,
                                            ptx::desc_at(d_v, hh * kHalf + kk * 2048), id_pv, 1);
                    ptx::mma_commit(bar(B_OF));
                    release(load_v(i));
                }
                __syncwarp();
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ MMA issue: the state's update
            const uint32_t id_mn = ptx::idesc_bf16_bmn(kC, kC);
            bool ok = true;
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const int valid = min(kC, len - (c0 + i) * kC);
                const uint64_t d_kt = ptx::desc_mnmajor_sw128(slot(load_k(i)), kHalf, 1024);
                if (!(ok = arrived(load_k(i), 18))) break;
                // (Q K^T may read these rows meanwhile: their scores are behind the diagonal, and not used.)
                if (valid < kC) zero_rows(smem + (load_k(i) % kSlots) * kTile, valid, lane);
                // Three parts each.  The first product overwrites the last chunk's update, so both halves of the
                // state warps have to have read that: they hand over w v after it.  16 tokens at a time, two
                // buffers for each half, so that one is formed while the other is multiplied.  The state-only
                // launch has a buffer for each 32 tokens, and two for the update (the tokens that the state
                // warps form come first: they have read the last but one).
                constexpr int kSteps = kState ? 4 : 8, kInner = kState ? 2 : 1;
#pragma unroll 1
                for (int e = 0; e < kSteps && ok; ++e) {
                    const int t = kState ? (e + 2) & 3 : e;               // tokens 32 t .. or 16 t ..
                    const int s = kState ? t : 2 * (e & 1) + (e >> 1 & 1);   // the buffer
                    const uint32_t use = kState ? (uint32_t)i : (uint32_t)(2 * i + (e >> 2));
                    if (!(ok = warp_wait(B_WF + s, use, 14))) break;
                    if (e == 0 && !(ok = warp_wait(B_WF + (kState ? 3 : 2), use, 17))) break;
                    if (ptx::elect_one()) {
                        ptx::tc_fence_after();
                        const uint32_t col = kState ? state_col_w(s) : kColW + s * 32;
#pragma unroll
                        for (int part = 0; part < 3; ++part)
#pragma unroll
                            for (int kk = 0; kk < kInner; ++kk)
                                ptx::mma_f16_ta(tmem + (kState ? state_col_d(i) : kColD), tmem + col + part * 8 * kInner + kk * 8,
                                                ptx::desc_at(d_kt, (kInner * t + kk) * 2048), id_mn, (e | part | kk) != 0);
                        ptx::mma_commit(bar(B_WE + s));
                        if (e == kSteps - 1) { // the state warps have read V before they handed over its last part
                            ptx::mma_commit(bar(B_DF + (i & 1)));
                            release(load_k(i));
                            release(load_v(i));
                        }
                    }
                    __syncwarp();
                }
            }
        } else {
            // ------------------------------------------------------------ gates
            constexpr int kGateWarps = kState ? 2 : 1;   // the state-only launch has a warp to spare, and less time
            const int gw = kState ? warp >> 1 : 0;
            double total[2] = {0.0, 0.0};
            float4 al[NH], be[NH];             // of tokens 4 lane .. 4 lane + 3
            auto fetch = [&](int i) {
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = (c0 + i) * kC + lane * 4 + e;
                        const size_t at = (size_t)(seq.x + t) * a.heads_v + head0 + h;
                        (&al[h].x)[e] = t < len ? __ldg(a.alpha + at) : 1.f;
                        (&be[h].x)[e] = t < len ? (a.beta ? __ldg(a.beta + at) : 1.f) : 0.f;   // weight zero past the end
                    }
            };
            if (gw < n) fetch(gw);
#pragma unroll 1
            for (int i = gw; i < n; i += kGateWarps) {
                if (i >= 2 && !warp_wait(B_GE + (i & 1), (uint32_t)((i >> 1) - 1), 30)) break;
                Gates &G = gates[i & 1];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    // One scan over the lanes, four tokens each; eight lanes are a block of 32 tokens.  (Four
                    // scans of 32 tokens, in a loop to save code, made this warp the slowest role.)
                    double L[4], sum = 0.0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float lg = log2f((&al[h].x)[e]);
                        sum += (double)(lg < kLogZero ? kLogZero : lg);   // a NaN stays one
                        L[e] = sum;
                    }
                    double scan = sum;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const double u = __shfl_up_sync(0xffffffffu, scan, d);
                        if (lane >= d) scan += u;
                    }
                    const double before = scan - sum, all = __shfl_sync(0xffffffffu, scan, 31);
                    const double end = __shfl_sync(0xffffffffu, scan, lane | 7);
                    const double prev = __shfl_sync(0xffffffffu, scan, max((lane & 24) - 1, 0));
                    const double start = lane < 8 ? 0.0 : prev;
                    const int quad = lane >> 2 & 3, J = lane & 3;
                    const double to = __shfl_sync(0xffffffffu, scan, max(8 * quad - 1, 0)), from = __shfl_sync(0xffffffffu, scan, 8 * J + 7);
                    if (lane < 16) G.step[h][quad][J] = (float)((quad ? to : 0.0) - (J == 3 ? 0.0 : from));
                    float4 rel, fac, w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const double Le = before + L[e];
                        const float beta = (&be[h].x)[e];
                        (&rel.x)[e] = (float)(Le - start);
                        (&fac.x)[e] = ptx::ex2_approx((float)(end - Le)) * beta;
                        (&w.x)[e] = exp2f((float)(all - Le)) * beta;
                    }
                    *reinterpret_cast<float4 *>(&G.rel[h][lane * 4]) = rel;
                    *reinterpret_cast<float4 *>(&G.fac[h][lane * 4]) = fac;
                    *reinterpret_cast<float4 *>(&G.w[h][lane * 4]) = w;
                    *reinterpret_cast<float4 *>(&G.beta[h][lane * 4]) = be[h];
                    if (lane == 0) G.all[h] = all;
                    total[h] += all;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_GF + (i & 1)));
                if (i + kGateWarps < n) fetch(i + kGateWarps);
            }
            if (kState && lane < 2) a.seg_log[((size_t)flat * (a.segments - 1) + seg) * 4 + gw * 2 + lane] = lane == 0 ? total[0] : total[1];
        }
    } else if (warp < 8) {
        // ---------------------------------------------------------------- P and O
        if (kState) {
            // These warps form w v of the first 64 tokens.
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int x = load_v(i);
                if (!warp_wait(B_GF + (i & 1), (uint32_t)(i >> 1), 50) || !warp_wait(B_F + x % kSlots, (uint32_t)(x / kSlots), 51)) break;
                bool ok = true;
#pragma unroll 1
                for (int s = 0; s < 2; ++s) {
                    if (i > 0 && !(ok = warp_wait(B_WE + s, (uint32_t)(i - 1), 52))) break;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int z = 0; z < 2; ++z) form(i, s * 32 + z * 16, state_col_w(s) + z * 8, 16);
                    formed();
                    if (lane == 0 && !(a.fault && i + s == 0)) ptx::mbar_arrive(bar(B_WF + s));
                }
                if (!ok) break;
                if (lane == 0) ptx::mbar_arrive(bar(B_GE + (i & 1)));
            }
        } else {
            const int quad = warp & 3, r = quad * 32 + lane;
            const uint32_t lanes = (uint32_t)(quad * 32) << 16;
            const uint32_t t_p = tmem + kColP + lanes, t_o = tmem + kColO + lanes;
            float skip[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) skip[h] = a.skip ? __ldg(a.skip + head0 + h) : 0.f;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const Gates &G = gates[i & 1];
                if (!both_wait(B_GF + (i & 1), (uint32_t)(i >> 1), B_SF, (uint32_t)i, 20)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int J = 0; J < 4; ++J) {  // 32 tokens j: read the scores, write P over them
                    uint32_t sv[32];
                    if (J <= quad) ptx::tmem_ld32(t_p + J * 32, sv);
                    const auto score = [&](int j) { return make_float2(__uint_as_float(sv[j]), __uint_as_float(sv[j + 1])); };
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        uint32_t pk[16];
                        const float rel = G.rel[h][r];
                        if (J < quad) {
                            // L_i less L at the end of block J.
                            const float row = ptx::ex2_approx(G.step[h][quad][J] + rel);
                            const float2 row2 = make_float2(row, row);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 f = *reinterpret_cast<const float4 *>(&G.fac[h][J * 32 + 4 * e]);
                                const float2 x = ptx::fmul2(score(4 * e), ptx::fmul2(row2, make_float2(f.x, f.y)));
                                const float2 y = ptx::fmul2(score(4 * e + 2), ptx::fmul2(row2, make_float2(f.z, f.w)));
                                pk[2 * e] = pack2(x.x, x.y);
                                pk[2 * e + 1] = pack2(y.x, y.y);
                            }
                        } else if (J == quad) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 rj = *reinterpret_cast<const float4 *>(&G.rel[h][J * 32 + 4 * e]);
                                const float4 bj = *reinterpret_cast<const float4 *>(&G.beta[h][J * 32 + 4 * e]);
                                float p[4];
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const int j = 4 * e + u;
                                    const float f = ptx::ex2_approx(rel - (&rj.x)[u]) * (&bj.x)[u];
                                    p[u] = j <= lane ? fmaf(__uint_as_float(sv[j]), f, j == lane ? skip[h] : 0.f) : 0.f;
                                }
                                pk[2 * e] = pack2(p[0], p[1]);
                                pk[2 * e + 1] = pack2(p[2], p[3]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[e] = 0u;
                        }
                        ptx::tmem_st16(t_p + J * 32 + h * 16, pk);
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_GE + (i & 1)));
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0 && !(a.fault && i == 0)) ptx::mbar_arrive(bar(B_PF));
                // The output of token r, half a row at a time: by way of shared memory to global memory in
                // one copy of the warp's 32 rows.  (16-byte stores from the lanes took five times as long, and
                // a bulk copy for each row as long as those.)  Rows past the sequence's end are another's: the
                // last chunk's rows are stored by their lanes.
                if (!warp_wait(B_OF, (uint32_t)i, 23)) break;
                ptx::tc_fence_after();
                const int t = (c0 + i) * kC + r, t_warp = (c0 + i) * kC + quad * 32;
#pragma unroll 1
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t out[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t ov[32];
                        ptx::tmem_ld32(t_o + hh * 64 + c * 32, ov);
#pragma unroll
                        for (int e = 0; e < 16; ++e) out[c * 16 + e] = pack2(__uint_as_float(ov[2 * e]), __uint_as_float(ov[2 * e + 1]));
                    }
                    if (hh == 1) {             // O's columns are free for the next chunk
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(B_OE));
                    }
                    if (t_warp + 32 <= len) {
                        uint8_t *mine = stage + quad * 4096;
                        if (lane == 0) ptx::bulk_wait_read_all();   // the rows before have left
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *reinterpret_cast<uint4 *>(mine + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                                make_uint4(out[4 * c], out[4 * c + 1], out[4 * c + 2], out[4 * c + 3]);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            ptx::tma_store_3d(&tm_o, hh * 64, item, seq.x + t_warp, ptx::smem_u32(mine));
                            ptx::bulk_commit();
                        }
                    } else if (t < len) {
                        __nv_bfloat16 *dst = a.o + ((size_t)(seq.x + t) * a.per_seq + item) * kC + hh * 64;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            reinterpret_cast<uint4 *>(dst)[c] = make_uint4(out[4 * c], out[4 * c + 1], out[4 * c + 2], out[4 * c + 3]);
                    }
                }
            }
            if (lane == 0) ptx::bulk_wait_read_all();   // before the CTA's shared memory goes
        }
    } else {
        // ---------------------------------------------------------------- the state
        const int wg = (warp >> 2) - 2, quad = warp & 3, r = quad * 32 + lane;   // row r of S, columns 64 wg ..
        const int h = NH == 2 ? r / kDv : 0;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        float st[64];
        // 32 rows x 64 columns of a warp, between global memory and a row per lane, by way of shared memory (the
        // copy's room, 4 KB a warp): half of the columns at a time, an access takes four rows' 128 bytes.
        // (Row by row a lane, each access touched 32 lines: 4.4 us to read a state and 4 to write it.)
        uint8_t *const mine = sop + (warp - 8) * 4096;
        const int row4 = lane >> 3, col4 = lane & 7;
        const auto far = [&](int k) { return (size_t)((k * 4 + row4) * kC + col4 * 4); };
        const auto near = [&](int row, int c) { return reinterpret_cast<float4 *>(mine + row * 128 + ((c ^ (row & 7)) << 4)); };
        auto store = [&](float *p) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float *from = st + half * 32 + c * 4;
                    *near(lane, c) = make_float4(from[0], from[1], from[2], from[3]);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) *reinterpret_cast<float4 *>(p + half * 32 + far(k)) = *near(k * 4 + row4, col4);
                __syncwarp();
            }
        };
        const size_t at = ((size_t)flat * kC + quad * 32) * kC + wg * 64;   // [batch, heads_v, dv] rows are flat 128-row items
        float *const slots = a.segments > 1 ? a.seg_state + ((size_t)flat * (a.segments - 1) * kC + quad * 32) * kC + wg * 64 : nullptr;
#pragma unroll
        for (int e = 0; e < 64; ++e) st[e] = 0.f;
        if (!kState) {
            // S0, or the first segment's state (S0 is in it) folded with those between: in the order of the loads,
            // which depend on nothing, then once into rows.  (By way of rows for each: 3 us a segment.)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float4 sum[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                const float *p = seg > 0 ? slots : a.S0 ? a.S0 + at : nullptr;
                if (p)
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum[k] = *reinterpret_cast<const float4 *>(p + half * 32 + far(k));
#pragma unroll 1
                for (int s = 1; s < seg; ++s) {
                    const double *lg = a.seg_log + ((size_t)flat * (a.segments - 1) + s) * 4 + h;
                    float4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = *reinterpret_cast<const float4 *>(slots + (size_t)s * kC * kC + half * 32 + far(k));
                    const float f = exp2f((float)(lg[0] + lg[2]));
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        sum[k] = make_float4(fmaf(f, sum[k].x, x[k].x), fmaf(f, sum[k].y, x[k].y), fmaf(f, sum[k].z, x[k].z),
                                             fmaf(f, sum[k].w, x[k].w));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) *near(k * 4 + row4, col4) = sum[k];
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 y = *near(lane, c);
                    float *to = st + half * 32 + c * 4;
                    to[0] = y.x;
                    to[1] = y.y;
                    to[2] = y.z;
                    to[3] = y.w;
                }
                __syncwarp();
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");   // the copy's room is free
        }
        // The bf16 copy that the next Q S^T reads: row r of this half.
        auto copy_out = [&] {
            uint8_t *dst = sop + wg * kHalf + r * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4 *>(dst + ((c ^ (r & 7)) << 4)) =
                    make_uint4(pack2(st[8 * c], st[8 * c + 1]), pack2(st[8 * c + 2], st[8 * c + 3]),
                               pack2(st[8 * c + 4], st[8 * c + 5]), pack2(st[8 * c + 6], st[8 * c + 7]));
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_SOP));
        };
        // S' = decay S + the update in these columns.
        auto take = [&](float decay, uint32_t col) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t d[32];
                ptx::tmem_ld32(tmem + col + wg * 64 + c * 32 + lanes, d);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 x = ptx::ffma2(make_float2(decay, decay), make_float2(st[c * 32 + e], st[c * 32 + e + 1]),
                                                make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1])));
                    st[c * 32 + e] = x.x;
                    st[c * 32 + e + 1] = x.y;
                }
            }
        };
        const uint32_t t_o = tmem + kColO + wg * 64 + lanes;
        const int ho = NH == 2 ? wg : 0;       // head of these output columns
        bool run = true;
        float decay = 0.f;
#pragma unroll 1
        for (int i = 0; i < n + (kState ? 1 : 0); ++i) {
            const int x = load_v(i);
            if (kState) {
                // Chunk i is formed before chunk i - 1 is taken, so that the tensor cores always have work.
                float next = 0.f;
                if (i < n) {
                    if (!(run = warp_wait(B_GF + (i & 1), (uint32_t)(i >> 1), 40) && warp_wait(B_F + x % kSlots, (uint32_t)(x / kSlots), 41) &&
                                (i == 0 || warp_wait(B_WE + 2 + wg, (uint32_t)(i - 1), 42))))
                        break;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int z = 0; z < 2; ++z) form(i, (2 + wg) * 32 + z * 16, state_col_w(2 + wg) + z * 8, 16);
                    formed();
                    if (lane == 0) ptx::mbar_arrive(bar(B_WF + 2 + wg));
                    next = exp2f((float)gates[i & 1].all[h]);
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(B_GE + (i & 1)));
                }
                if (i > 0) {
                    if (!(run = warp_wait(B_DF + ((i - 1) & 1), (uint32_t)((i - 1) >> 1), 43))) break;
                    ptx::tc_fence_after();
                    take(decay, state_col_d(i - 1));
                }
                decay = next;
                continue;
            }
            copy_out();                        // Q S^T of the last chunk was issued before its update was done
            if (!(run = both_wait(B_GF + (i & 1), (uint32_t)(i >> 1), B_F + x % kSlots, (uint32_t)(x / kSlots), 40))) break;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const int mine = 2 * wg + (j & 1), uses = 2 * i + (j >> 1);
                if (uses > 0 && !(run = warp_wait(B_WE + mine, (uint32_t)(uses - 1), 42))) break;
                ptx::tc_fence_after();
                form(i, (2 * j + wg) * 16, kColW + mine * 32, 8);
                formed();
                if (lane == 0) ptx::mbar_arrive(bar(B_WF + mine));
            }
            if (!run) break;
            const Gates &G = gates[i & 1];
            decay = exp2f((float)G.all[h]);
            const float gamma = ptx::ex2_approx(G.step[ho][quad][3] + G.rel[ho][r]);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_GE + (i & 1)));
            // diag(2^L) Q S^T, onto which P V is added: token r, these columns.
            if (!(run = warp_wait(B_OQ, (uint32_t)i, 44))) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t ov[16];
                float of[16];
                ptx::tmem_ld16(t_o + c * 16, of);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 x = ptx::fmul2(make_float2(gamma, gamma), make_float2(of[e], of[e + 1]));
                    ov[e] = __float_as_uint(x.x);
                    ov[e + 1] = __float_as_uint(x.y);
                }
                ptx::tmem_st16(t_o + c * 16, ov);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_PF));
            if (!(run = warp_wait(B_DF + (i & 1), (uint32_t)(i >> 1), 43))) break;
            ptx::tc_fence_after();
            take(decay, kColD);
        }
        float *dst = kState || beside ? slots + (size_t)seg * kC * kC : last && a.S_new ? a.S_new + at : nullptr;
        if (dst && run) store(dst);        // the last Q S^T has read its copy
    }

    // -------------------------------------------------------------------- teardown
    ptx::tc_fence_before();
    __syncthreads();                           // all roles have ended: `aborted` no longer changes
    if (aborted) {
        if (tid == 0 && a.err) latch_error(a.err, STREE_ERR_TIMEOUT, b, aborted, 0);
        if ((warp == 1 || warp == 2) && ptx::elect_one()) {
            ptx::mma_commit(bar(B_DRAIN + warp - 1));   // every issued MMA completes first
            ptx::mbar_wait(bar(B_DRAIN + warp - 1), 0);
        }
        // Copies that may still land (`loads`: the producer's lane).
#pragma unroll 1
        for (int x = max(0, loads - kSlots); x < loads; ++x) ptx::mbar_wait(bar(B_F + x % kSlots), (uint32_t)((x / kSlots) & 1));
        ptx::tc_fence_before();
        __syncthreads();
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    if (beside) wait_dependency();         // what follows this launch follows the state-only one too
}

std::mutex g_mutex;
int g_sms[kMaxDevices] = {};

cudaError_t prepare(int *sms)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_sms[dev]) {
        const auto set = [](auto *f) { return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem); };
        if ((e = set(linear_tc_kernel<1, false>)) != cudaSuccess || (e = set(linear_tc_kernel<2, false>)) != cudaSuccess ||
            (e = set(linear_tc_kernel<1, true>)) != cudaSuccess || (e = set(linear_tc_kernel<2, true>)) != cudaSuccess)
            return e;
        int n = 0;
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        g_sms[dev] = n > 0 ? n : 1;
    }
    *sms = g_sms[dev];
    return cudaSuccess;
}

// Segments of a sequence: as many as fill the SMs with one CTA each in both passes, while a segment of a
// sequence of average length has at least four chunks (a CTA's set-up and the first launch
// cost about two).
int segments_for(int batch, int total, int items, int sms)
{
    int s = sms / (items > 0 ? items : 1);
    const int by_len = total / (batch > 0 ? batch : 1) / (4 * kC);
    s = s < by_len ? s : by_len;
    return s < 2 ? 1 : s + 1 > kMaxSegments ? kMaxSegments : s + 1;   // the first runs beside the states
}

size_t workspace_for(int items, int segments)
{
    return segments > 1 ? (size_t)items * (segments - 1) * (kC * kC * sizeof(float) + 4 * sizeof(double)) : 0;
}

}  // namespace

bool linear_tc_supported(int heads_v, int heads_k, int dk, int dv, stree_dtype dtype)
{
    return dtype == STREE_BF16 && dk == kC && (dv == kC || (dv == kC / 2 && (heads_v / heads_k) % 2 == 0));
}

cudaError_t linear_tc_workspace(int batch, int total, int heads_v, int dv, size_t *bytes)
{
    int sms = 0;
    const cudaError_t e = prepare(&sms);
    if (e != cudaSuccess) return e;
    const int items = batch * (heads_v * dv / kC);
    *bytes = workspace_for(items, segments_for(batch, total, items, sms));
    return cudaSuccess;
}

cudaError_t launch_linear_tc(const LinearArgs &l, void *workspace, size_t workspace_bytes, cudaStream_t s)
{
    int sms = 0;
    cudaError_t e = prepare(&sms);
    if (e != cudaSuccess) return e;
    TcArgs a{};
    a.alpha = l.alpha;
    a.beta = l.beta;
    a.skip = l.skip;
    a.S0 = l.S0;
    a.cu = l.cu;
    a.o = static_cast<__nv_bfloat16 *>(l.o);
    a.S_new = l.S_new;
    a.err = l.err;
    a.total = l.total;
    a.batch = l.batch;
    a.heads_v = l.heads_v;
    a.heads_k = l.heads_k;
    a.per_seq = l.heads_v * l.dv / kC;
    const WaitHook hook = wait_hook();
    a.wait_ns = hook.limit_ns;
    a.fault = hook.fault;
    const int items = l.batch * a.per_seq;
    a.segments = segments_for(l.batch, l.total, items, sms);
    if (!workspace || workspace_bytes < workspace_for(items, a.segments)) a.segments = 1;
    if (a.segments > 1) {
        a.seg_log = static_cast<double *>(workspace);
        a.seg_state = reinterpret_cast<float *>(a.seg_log + (size_t)items * (a.segments - 1) * 4);
    }
    CUtensorMap q{}, k{}, v{}, o{};
    if (l.total > 0 && (!encode_heads(&q, l.q, l.total, l.heads_k, 1, kC) || !encode_heads(&k, l.k, l.total, l.heads_k, 1, kC) ||
                        !encode_heads(&v, l.v, l.total, a.per_seq, 1, kC) || !encode_heads(&o, l.o, l.total, a.per_seq, 1, 32)))
        return cudaErrorInvalidValue;
    const bool one = l.dv == kC;
    const auto walk = [&](int first, int count) {
        a.seg_first = first;
        a.seg_count = count;
        const dim3 grid((unsigned)(items * count + (a.segments == 1 ? 1 : 0)));   // and the error word
        return one ? launch_pdl(linear_tc_kernel<1, false>, grid, kThreads, kSmem, s, q, k, v, o, a)
                   : launch_pdl(linear_tc_kernel<2, false>, grid, kThreads, kSmem, s, q, k, v, o, a);
    };
    if (a.segments == 1) return walk(0, 1);
    a.seg_first = 1;
    a.seg_count = a.segments - 2;
    const dim3 grid((unsigned)(items * a.seg_count + 1));   // and the error word
    e = one ? launch_pdl(linear_tc_kernel<1, true>, grid, kThreads, kSmem, s, q, k, v, o, a)
            : launch_pdl(linear_tc_kernel<2, true>, grid, kThreads, kSmem, s, q, k, v, o, a);
    if (e != cudaSuccess || (e = walk(0, 1)) != cudaSuccess) return e;
    return walk(1, a.segments - 1);
}

}  // namespace stree
