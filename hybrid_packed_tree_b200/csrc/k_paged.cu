// k_paged.cu -- attention of one new token per sequence over a paged key-value cache,
// split over the cache's length and joined, sm_100a.
//
//   o[b,h] = sum_j softmax_j(scale q[b,h] . k_j) v_j,  j in [0, len_b), k_j and v_j in
//   page table[b][j / page_size] at row j % page_size of key/value head h / (Hq / Hkv).
//
// One new token makes 4 d flops per query head and cached byte pair: far below what the
// tensor cores need to be busy, so the kernel is bound by HBM and everything serves the
// loads.  The keys and values of every (sequence, key/value head, 16 query heads of the
// group) are a row of blocks of 64 positions; the blocks of all rows form one list, cut
// into equal contiguous shares, one per CTA (two CTAs per SM), so ragged lengths, one
// long sequence and many short ones all load the SMs evenly.  A producer warp fetches the
// page ids one block ahead and issues one TMA box per run of rows inside a page (at most
// sixteen per block, each lane its own) into a ring of stages; four warps take a quarter of
// the block each (16 positions, 32 with 8-bit pages), with their own running maximum, sum and output (one pass, online
// softmax), and are joined in shared memory where the share leaves a row of blocks.  A row
// of blocks that lies in one share is finished there; the pieces of the others go to the
// workspace and a second launch joins them by the log-sum-exp rule.
//
// The products run on the warp-level matrix instruction.  K Q^T: 16 keys are its rows and eight
// query heads its columns.  V^T P: 16 value columns are its rows, the heads its columns again.  K and V
// arrive by ldmatrix straight from the swizzled tile; the probabilities stay in registers and are
// turned into the second product's operand by a transposing move.  A 128-row tcgen05 tile of query heads
// would be at most one eighth full and adds a round trip through tensor memory for each block.
// 8-bit pages: keys and values become fp16 exactly (every e4m3 is one).  A query row is
// scaled to [-2^15, 2^15] by a power of two so that it is fp16 as well, exactly down to 2^-31 of
// the row's largest element (below, to 2^-40 of it; scaled to [-1, 1], elements below 2^-16 lost bits that
// decide a score where the keys are zero in the strong channels).  A key's scale
// multiplies its score; a value's scale 2^e joins its probability before that is rounded to
// fp16, so the sum has a reference of its own, the maximum of score + e less 15: the largest weight is
// 2^15, none overflows whatever the scales, and a weight has fp16's eleven bits down to 2^-29 of the largest
// and is gone below 2^-40.  (With a largest weight of 1 those were 2^-14 and 2^-25: a key that takes nearly all
// of the softmax with a value near zero left nothing of the others.)  (Values widened to bf16 with the scale on a bf16
// probability: 120 us; so and with page positions followed without divisions 93; with the keys
// and not 16 query heads as the instruction's rows 60.)
//
// Measured, calls one behind the other on changing inputs: one sequence of 131065 tokens, bf16, 32 heads over 8
// (537 MB): 94 us a call, 82 of them this kernel's (6.5 TB/s, a copy's rate) and the rest the join's; 64 sequences of
// up to 4096 tokens, e4m3 (272 MB): 68 us, with 53 % of DRAM and 45 % of the issue slots in use: the chain of a
// block's steps in each warp (conversion, scores, maxima, exponentials, conversion, values) and the join.
#include <cuda.h>

#include <mutex>

#include "seq_pages.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace stree {

stree_status check_cache(const void *k_pages, const void *v_pages, const void *k_scales, const void *v_scales,
                         const int32_t *table, int batch, int heads_kv, int head_dim, int n_pages, int page_size,
                         int max_pages, stree_dtype cache);

namespace {

constexpr int kD = kCacheDim;
constexpr int kComputeWarps = 4;
// Positions per block: 16 for each warp, 32 with 8-bit pages, where the work on a position counts
// more than its bytes (two tiles share a maximum and hide each other's latencies).
__host__ __device__ constexpr int block_positions(bool e4m3) { return e4m3 ? 128 : 64; }
constexpr int kThreads = (kComputeWarps + 1) * 32;
constexpr int kMaxHeads = 16;                  // query heads in a row of blocks
constexpr int kJoinRow = kD + 4;               // floats of a row in shared memory (no bank conflicts)
constexpr int kMaxStages = 8;
constexpr int kLift = 15;                      // 8-bit pages: log2 of the largest scaled query element and weight

constexpr int kCtasPerSm = 2;
constexpr int kSmemPerCta = 226 * 1024 / kCtasPerSm;
constexpr int kCombineWarps = 16, kCombineThreads = kCombineWarps * 32;

struct PagedArgs {
    const __nv_bfloat16 *q;
    const uint8_t *k_scales, *v_scales;
    const int32_t *table, *lens;
    __nv_bfloat16 *o;
    float *part_o;                             // [share][2][rows][128]
    float4 *part_ml;                           // [share][2][rows]: (output's reference, sum's reference, sum,
                                               // nonzero: a page out of range)
    int *gave_up;                              // [share]: the wait that ran out there, or 0; the join reports it.  (The
                                               // shares cannot: the word is cleared by a block that starts when the
                                               // first of them have ended.)
    int32_t *err;
    int batch, heads_q, heads_kv, group, row_tiles, rows;   // rows: min(group, 16)
    int n_pages, page_size, max_pages, blk, box_rows, shares, stages;   // blk: positions per block
    float scale_log2;
    uint32_t wait_ns;                          // limit of a wait
    int fault;                                 // test hook: 1 withholds a share's first block
};

__device__ __forceinline__ int blocks_of(const PagedArgs &a, int b)
{
    const int n = min(max(__ldg(a.lens + b), 0), a.max_pages * a.page_size);
    return (n + a.blk - 1) / a.blk;
}

__device__ __forceinline__ long long share_begin(long long total, int c, int shares) { return total * c / shares; }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Joins partial results (output's reference, sum's reference, sum) whose outputs and sums are
// x = 2^-reference (unnormalised output) and likewise the sum.
__device__ __forceinline__ float weight(float ref, float top) { return ref == -INFINITY ? 0.f : ptx::ex2_approx(ref - top); }

// Output over sum, given both references.
__device__ __forceinline__ float quotient(float x, float ref, float m, float sum)
{
    return sum > 0.f ? x * ptx::ex2_approx(ref - m) / sum : x;
}

// The transpose of an 8 x 8 tile of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

struct Stage {                                 // offsets inside a stage of the ring
    uint32_t k, v, ks, vs, bytes;
};

template <bool kE4m3>
__host__ __device__ constexpr Stage stage_layout()
{
    // 8-bit pages: [128][128 B] tiles and 128 scale bytes each; bf16: [64] rows, two 64-column halves.
    return kE4m3 ? Stage{0, 16384, 32768, 32768 + 128, 32768 + 1024} : Stage{0, 16384, 0, 0, 32768};
}

// What the compute warps do together when a wait of the CTA has run out (the producer gives up
// too then).  Out of line: inlined it cost the loop registers (bf16, 32 heads over 2: 43 us against 41.3).
__device__ __noinline__ void give_up(int *report, int where, uint32_t produced, const volatile int *issued_s, uint32_t full0,
                                     int stages, int fault, float4 *piece, int rows)
{
    const int tid = threadIdx.x;
    ptx::mbar_wait(produced, 0);
    if (tid == 0) {
        *report = where;
        // Nothing may still be landing in shared memory when the CTA ends.
        const int issued = *issued_s;
        for (int i = max(fault, issued - stages); i < issued; ++i)
            ptx::mbar_wait(full0 + 8 * (i % stages), (uint32_t)((i / stages) & 1));
    }
    // The join leaves rows alone that have a piece in this share.
    for (int e = tid; e < 2 * rows; e += kComputeWarps * 32) piece[e] = make_float4(0.f, 0.f, 0.f, 1.f);
}

// NT: tiles of eight query heads in a row of blocks.
template <bool kE4m3, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
paged_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const PagedArgs a)
{
    constexpr Stage L = stage_layout<kE4m3>();
    constexpr int kHeads = 8 * NT, kBlk = block_positions(kE4m3), KT = kBlk / 64;   // KT: tiles of 16 positions a warp
    constexpr int kEighths = kBlk / 8;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bars[2 * kMaxStages + 1];
    __shared__ int tmp[33], found[2];
    __shared__ volatile int aborted, issued_s, bad[kMaxStages];
    __shared__ float4 ml_s[kComputeWarps][kHeads];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    float *joined = reinterpret_cast<float *>(smem + a.stages * L.bytes);   // [4][rows][132]
    auto full = [&](int s) { return ptx::smem_u32(&bars[s]); };
    auto empty = [&](int s) { return ptx::smem_u32(&bars[kMaxStages + s]); };
    const uint32_t produced = ptx::smem_u32(&bars[2 * kMaxStages]);   // the producer has ended
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    pdl_start();
    if (blockIdx.x == a.shares) {              // the error word
        PageCheck c{};
        c.count = a.lens;
        c.table = a.table;
        c.batch = a.batch;
        c.n_pages = a.n_pages;
        c.page_size = a.page_size;
        c.max_pages = a.max_pages;
        c.clamp = a.max_pages * a.page_size;
        check_pages(c, a.err);
        return;
    }
    // Rows of sequences with no position are zero.
    for (int b = blockIdx.x; b < a.batch; b += a.shares)
        if (blocks_of(a, b) == 0)
            for (int e = tid; e < a.heads_q * kD / 8; e += kThreads)
                reinterpret_cast<uint4 *>(a.o + (size_t)b * a.heads_q * kD)[e] = make_uint4(0u, 0u, 0u, 0u);
    // This CTA's share of the list.
    const int per_seq = a.heads_kv * a.row_tiles;
    int n_all = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        int t;
        block_scan(b0 + tid < a.batch ? blocks_of(a, b0 + tid) : 0, tmp, &t);
        n_all += t;
    }
    const long long total = (long long)n_all * per_seq;
    const int shares = (int)min((long long)a.shares, total);   // no share is empty
    if ((int)blockIdx.x >= shares) {
        if (tid == 0) a.gave_up[blockIdx.x] = 0;
        return;
    }
    const long long begin = share_begin(total, blockIdx.x, shares), end = share_begin(total, blockIdx.x + 1, shares);
    // The list is ordered by sequence, then by (key/value head, row tile), then by block.
    block_find(a.batch, (int)(begin / per_seq), [&](int b) { return blocks_of(a, b); }, tmp, found);
    const int b_first = found[0];
    const long long seq_at = (long long)found[1] * per_seq;

    if (tid == 0) {
        for (int s = 0; s < a.stages; ++s) {
            ptx::mbar_init(full(s), kE4m3 ? 1 + 2 * kEighths : 1);
            ptx::mbar_init(empty(s), kComputeWarps);
        }
        ptx::mbar_init(produced, 1);
        ptx::fence_mbar_init();
        aborted = 0;
    }
    __syncthreads();

    // Where the share begins: its sequence, row of blocks (item) and block.
    int b = b_first, nb = blocks_of(a, b);
    long long left = end - begin;
    int item = (int)((begin - seq_at) / nb), blk = (int)((begin - seq_at) % nb);
    auto advance = [&] {                       // to the next block of the list
        if (++blk < nb) return;
        blk = 0;
        if (++item < per_seq) return;
        item = 0;
        do ++b;
        while (b < a.batch && (nb = blocks_of(a, b)) == 0);
    };

    if (warp == kComputeWarps) {
        // ------------------------------------------------------------ producer
        const int boxes = kBlk / a.box_rows;
        const uint32_t box_bytes = (uint32_t)a.box_rows * 128u;
        if (lane == 0) {
            ptx::prefetch_tensormap(&tm_k);
            ptx::prefetch_tensormap(&tm_v);
        }
        // Lane i (mod the block's eighths) follows positions 8 i .. 8 i + 7 of the block (an eighth lies in one page): their
        // page's place in the table and row in the page, moved on by a block without a
        // division (the page ids of one block ahead are in flight while a block is issued).
        const int mine8 = (lane & (kEighths - 1)) * 8, step_p = kBlk / a.page_size, step_r = kBlk % a.page_size;
        const int first_p = mine8 / a.page_size, first_r = mine8 % a.page_size;
        int at_p = (blk * kBlk + mine8) / a.page_size, at_r = (blk * kBlk + mine8) % a.page_size;
        int n = min(max(__ldg(a.lens + b), 0), a.max_pages * a.page_size);
        int row0 = a.row_tiles == 1 ? item : item / a.row_tiles;   // key/value head
        auto lookup = [&]() -> int {
            if (blk * kBlk + mine8 >= n) return -2;   // nothing there
            return __ldg(a.table + (size_t)b * a.max_pages + at_p);
        };
        int id = lookup(), stage = 0, issued = 0;
        uint32_t lap = 0;                      // how often the ring has been filled
#pragma unroll 1
        for (; left > 0; --left, ++issued) {
            const int chead = row0, crow = at_r;
            const int cid = id == -2 || (id >= 0 && id < a.n_pages) ? id : -1;
            if (left > 1) {
                const int was_b = b, was_item = item;
                advance();
                if (b != was_b || item != was_item) {
                    at_p = first_p;
                    at_r = first_r;
                    row0 = a.row_tiles == 1 ? item : item / a.row_tiles;
                    if (b != was_b) n = min(max(__ldg(a.lens + b), 0), a.max_pages * a.page_size);
                } else {
                    at_p += step_p;
                    at_r += step_r;
                    if (at_r >= a.page_size) {
                        at_r -= a.page_size;
                        ++at_p;
                    }
                }
                id = lookup();
            }
            if (lap > 0 && !wait_warp(&aborted, empty(stage), lap - 1, 1, a.wait_ns)) break;
            const int eighth = (lane * (a.box_rows / 8)) & (kEighths - 1);   // of the box that this lane issues
            const int box_id = __shfl_sync(0xffffffffu, cid, eighth), box_row = __shfl_sync(0xffffffffu, crow, eighth);
            const bool given = !(a.fault && issued == 0);
            const bool mine = lane < boxes && box_id >= 0 && given;
            const uint32_t n_boxes = __popc(__ballot_sync(0xffffffffu, mine));
            const bool any_bad = __any_sync(0xffffffffu, cid == -1);
            const uint32_t base = ptx::smem_u32(smem) + stage * L.bytes, fb = full(stage);
            if (lane == 0 && given) {
                bad[stage] = any_bad;
                ptx::mbar_expect_tx(fb, n_boxes * box_bytes * (kE4m3 ? 2u : 4u));
            }
            __syncwarp();
            if (mine) {
                const int row = (box_id * a.heads_kv + chead) * a.page_size + box_row;
                const uint32_t at = base + (uint32_t)lane * box_bytes;
                ptx::tma_load_2d(at + L.k, &tm_k, 0, row, fb);
                ptx::tma_load_2d(at + L.v, &tm_v, 0, row, fb);
                if (!kE4m3) {
                    ptx::tma_load_2d(at + L.k + 8192, &tm_k, 64, row, fb);
                    ptx::tma_load_2d(at + L.v + 8192, &tm_v, 64, row, fb);
                }
            }
            if (kE4m3 && given) {
                // Half the lanes the eighths of the key scales, half of the value scales.
                if (cid >= 0)
                    ptx::cp_async8(base + (lane < kEighths ? L.ks : L.vs) + mine8,
                                   (lane < kEighths ? a.k_scales : a.v_scales) + ((size_t)cid * a.heads_kv + chead) * a.page_size + crow);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
            }
            if (++stage == a.stages) {
                stage = 0;
                ++lap;
            }
        }
        __syncwarp();
        if (lane == 0) {
            issued_s = issued;
            ptx::mbar_arrive(produced);
        }
        return;                                // early: with it waiting for the others the join's CTAs start late (44.8 us against 41.3)
    }

    // ---------------------------------------------------------------- compute
    const int t4 = lane & 3, r4 = lane >> 2;
    int s = 0;                                 // the stage, and its use's number
    uint32_t phase = 0;
    bool run = true;
    int piece = 0;                             // 0: the share's first row of blocks, 1: a later one
    while (left > 0 && run) {
        const int hkv = item / a.row_tiles, rt = item % a.row_tiles;
        const int head0 = hkv * a.group + rt * kHeads;
        const int rows = min(kHeads, a.group - rt * kHeads);
        const int cb = b, blk0 = blk, cnb = nb;
        const int n = min(max(__ldg(a.lens + cb), 0), a.max_pages * a.page_size);
        const bool whole = blk0 == 0 && left >= cnb;
        // Q as the B operand: head r4 (+ 8 for the second tile), zero past the group.  With 8-bit
        // pages the columns are permuted as the key bytes lie: k index 2 t, 2 t + 1 of a step is
        // column 4 t, 4 t + 1, and 2 t + 8, 2 t + 9 is 4 t + 2, 4 t + 3.
        uint32_t qf[NT][8][2];
        float qs[NT][2];                       // log2-scale of the scores of heads 2 t4, 2 t4 + 1
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int head = t * 8 + r4;
            const __nv_bfloat16 *qp = a.q + ((size_t)cb * a.heads_q + head0 + head) * kD;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = kE4m3 ? kk * 16 + t4 * 4 + i * 2 : kk * 16 + t4 * 2 + i * 8;
                    qf[t][kk][i] = head < rows ? __ldg(reinterpret_cast<const uint32_t *>(qp + col)) : 0u;
                }
            float f = a.scale_log2;
            if (kE4m3) {
                uint32_t top = 0;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) top = max(top, max(finite_top2(qf[t][kk][0]), finite_top2(qf[t][kk][1])));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // The row's largest magnitude lies in [2^(e-127), 2^(e-126)); both factors are normal numbers.
                const uint32_t e = max(top >> 7, (uint32_t)kLift);
                const float inv = power_of_two(253u + kLift - e);
                f *= power_of_two(e + 1u - kLift);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = qf[t][kk][i];
                        qf[t][kk][i] = pack_half(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xffff0000u) * inv);
                    }
            }
            qs[t][0] = __shfl_sync(0xffffffffu, f, t4 * 8);
            qs[t][1] = __shfl_sync(0xffffffffu, f, t4 * 8 + 4);
        }
        float acc[NT][8][4];                   // 16 columns a step: rows r4, r4 + 8 of the tile, heads 2 t4, 2 t4 + 1
        float m[NT][2], ref[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[t][c][j] = 0.f;
            m[t][0] = m[t][1] = ref[t][0] = ref[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
        }
        int any_bad = 0;
#pragma unroll 1
        while (true) {
            if (!(run = wait_warp(&aborted, full(s), phase, 10, a.wait_ns))) break;
            any_bad |= bad[s];
            const uint32_t base = ptx::smem_u32(smem) + s * L.bytes;
            const int key0 = warp * 16 * KT, valid = n - (blk * kBlk + key0);   // positions of this warp that exist
            if (valid > 0) {
                const bool tail = valid < 16 * KT;
                // Scores: keys r4, r4 + 8 of each 16 by heads 2 t4, 2 t4 + 1.
                float sc[KT][NT][4];
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int t = 0; t < NT; ++t) sc[u][t][0] = sc[u][t][1] = sc[u][t][2] = sc[u][t][3] = 0.f;
                // Tiles of eight keys by 16 bytes: keys 0-7 and 8-15 of a chunk, then of the next.
                const int krow = key0 + (lane & 15), ksw = krow & 7;
                const uint32_t kaddr = base + L.k + krow * 128, vaddr = base + L.v;
                if (kE4m3) {
#pragma unroll
                    for (int kk = 0; kk < 8; kk += 2)
#pragma unroll
                        for (int u = 0; u < KT; ++u) {
                            uint32_t r[4];
                            ldsm4(kaddr + u * 2048 + (((kk + (lane >> 4)) ^ ksw) << 4), r);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint32_t k[4];
                                e4m3x4_to_f16(r[2 * j], k[0], k[2]);
                                e4m3x4_to_f16(r[2 * j + 1], k[1], k[3]);
#pragma unroll
                                for (int t = 0; t < NT; ++t) mma16816<true>(sc[u][t], k, qf[t][kk + j][0], qf[t][kk + j][1]);
                            }
                        }
                } else {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        uint32_t r[4];
                        const int chunk = kk * 2 + (lane >> 4);
                        ldsm4(kaddr + (chunk >> 3) * 8192 + (((chunk & 7) ^ ksw) << 4), r);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16816<false>(sc[0][t], r, qf[t][kk][0], qf[t][kk][1]);
                    }
                }
                float kf[KT][2], ve[KT][2];    // a key's scale, log2 of a value's
#pragma unroll
                for (int u = 0; u < KT; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        kf[u][j] = 1.f;
                        ve[u][j] = 0.f;
                        if (kE4m3) {
                            const uint8_t *sb = smem + s * L.bytes + key0 + 16 * u + 8 * j + r4;
                            kf[u][j] = power_of_two(sb[L.ks]);
                            ve[u][j] = __uint_as_float(0x4b000000u | sb[L.vs]) - 8388735.f;   // 2^23 + byte, less 2^23 + 127
                        }
                    }
                uint32_t pf[KT][NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int u = 0; u < KT; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sc[u][t][e] *= kE4m3 ? qs[t][e & 1] * kf[u][e >> 1] : qs[t][e & 1];
                            if (tail && 16 * u + 8 * (e >> 1) + r4 >= valid) sc[u][t][e] = -INFINITY;
                        }
                    // Running maxima of the scores and, for the output, of the scores with the values' scales.
                    float mn[2], rn[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mn[i] = fmaxf(sc[0][t][i], sc[0][t][2 + i]);
                        rn[i] = fmaxf(sc[0][t][i] + ve[0][0], sc[0][t][2 + i] + ve[0][1]);
#pragma unroll
                        for (int u = 1; u < KT; ++u) {
                            mn[i] = fmaxf(mn[i], fmaxf(sc[u][t][i], sc[u][t][2 + i]));
                            rn[i] = fmaxf(rn[i], fmaxf(sc[u][t][i] + ve[u][0], sc[u][t][2 + i] + ve[u][1]));
                        }
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            mn[i] = fmaxf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], d));
                            if (kE4m3) rn[i] = fmaxf(rn[i], __shfl_xor_sync(0xffffffffu, rn[i], d));
                        }
                        mn[i] = fmaxf(m[t][i], mn[i]);
                        rn[i] = kE4m3 ? fmaxf(ref[t][i], rn[i] - (float)kLift) : mn[i];
                    }
                    if (__any_sync(0xffffffffu, mn[0] > m[t][0] || mn[1] > m[t][1] || rn[0] > ref[t][0] || rn[1] > ref[t][1])) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float f = rn[i] == ref[t][i] ? 1.f : ptx::ex2_approx(ref[t][i] - rn[i]);
                            l[t][i] *= mn[i] == m[t][i] ? 1.f : ptx::ex2_approx(m[t][i] - mn[i]);
                            m[t][i] = mn[i];
                            ref[t][i] = rn[i];
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                acc[t][c][i] *= f;
                                acc[t][c][2 + i] *= f;
                            }
                        }
                    }
                    // Probabilities; turned from (key, head) to the B operand's (head, key) by a transposing move.
                    const float m0 = m[t][0] == -INFINITY ? 0.f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
                    const float r0 = ref[t][0] == -INFINITY ? 0.f : ref[t][0], r1 = ref[t][1] == -INFINITY ? 0.f : ref[t][1];
#pragma unroll
                    for (int u = 0; u < KT; ++u)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float s0 = sc[u][t][2 * j], s1 = sc[u][t][2 * j + 1];
                            const float p0 = ptx::ex2_approx(s0 - m0), p1 = ptx::ex2_approx(s1 - m1);
                            l[t][0] += p0;
                            l[t][1] += p1;
                            pf[u][t][j] = transpose8(kE4m3 ? pack_half(ptx::ex2_approx(s0 + (ve[u][j] - r0)), ptx::ex2_approx(s1 + (ve[u][j] - r1)))
                                                           : pack_bf16(p0, p1));
                        }
                }
                // Positions past the end hold anything: their value rows count as zero.
                auto keep = [&](int key) { return (key < valid ? 0xffffu : 0u) | (key + 1 < valid ? 0xffff0000u : 0u); };
                if (kE4m3) {
                    // A thread gets columns 2 r4, 2 r4 + 1 of keys 2 t4, 2 t4 + 1: the even columns are
                    // the operand's rows 0-7, the odd ones its rows 8-15.
#pragma unroll
                    for (int c = 0; c < 8; c += 2)
#pragma unroll
                        for (int u = 0; u < KT; ++u) {
                            uint32_t r[4];
                            ldsm4_t(vaddr + krow * 128 + u * 2048 + (((c + (lane >> 4)) ^ ksw) << 4), r);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint32_t v[4];
                                e4m3x4_to_f16(__byte_perm(r[2 * j], 0, 0x3120), v[0], v[1]);
                                e4m3x4_to_f16(__byte_perm(r[2 * j + 1], 0, 0x3120), v[2], v[3]);
                                if (tail) {
                                    v[0] &= keep(16 * u + 2 * t4);
                                    v[1] &= keep(16 * u + 2 * t4);
                                    v[2] &= keep(16 * u + 2 * t4 + 8);
                                    v[3] &= keep(16 * u + 2 * t4 + 8);
                                }
#pragma unroll
                                for (int t = 0; t < NT; ++t) mma16816<true>(acc[t][c + j], v, pf[u][t][0], pf[u][t][1]);
                            }
                        }
                } else {
                    // Tiles: keys 0-7 of two chunks of eight columns, then keys 8-15.
                    const int vrow = key0 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t v[4];
                        const int chunk = 2 * c + ((lane >> 3) & 1);
                        ldsm4_t(vaddr + (chunk >> 3) * 8192 + vrow * 128 + (((chunk & 7) ^ (vrow & 7)) << 4), v);
                        if (tail) {
                            v[0] &= keep(2 * t4);
                            v[1] &= keep(2 * t4);
                            v[2] &= keep(2 * t4 + 8);
                            v[3] &= keep(2 * t4 + 8);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16816<false>(acc[t][c], v, pf[0][t][0], pf[0][t][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty(s));
            if (++s == a.stages) {
                s = 0;
                ++phase;
            }
            --left;
            const bool last = left == 0 || blk + 1 == nb;
            if (left > 0) advance();
            if (last) break;
        }
        // Join the four warps: each leaves its rows, then a thread takes one column.  The lift ends here.
        constexpr float kLifted = kE4m3 ? (float)kLift : 0.f, kLower = kE4m3 ? 1.f / (1 << kLift) : 1.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], d);
                const int r = t * 8 + 2 * t4 + i;
                if (r >= rows) continue;
                if (r4 == 0) ml_s[warp][r] = make_float4(ref[t][i] + kLifted, m[t][i], l[t][i], 0.f);
                float *dst = joined + ((size_t)warp * a.rows + r) * kJoinRow;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (kE4m3) {
                        *reinterpret_cast<float2 *>(dst + 16 * c + 2 * r4) = make_float2(acc[t][c][i], acc[t][c][2 + i]);
                    } else {
                        dst[16 * c + r4] = acc[t][c][i];
                        dst[16 * c + 8 + r4] = acc[t][c][2 + i];
                    }
                }
            }
        asm volatile("bar.sync 1, %0;" ::"n"(kComputeWarps * 32) : "memory");
        if (!aborted) {
            const size_t slot = (size_t)blockIdx.x * 2 + piece;
            for (int r = 0; r < rows; ++r) {
                float R = -INFINITY, M = -INFINITY, den = 0.f, x = 0.f;
#pragma unroll
                for (int w = 0; w < kComputeWarps; ++w) {
                    R = fmaxf(R, ml_s[w][r].x);
                    M = fmaxf(M, ml_s[w][r].y);
                }
#pragma unroll
                for (int w = 0; w < kComputeWarps; ++w) {
                    const float4 ml = ml_s[w][r];
                    x = fmaf(weight(ml.x, R) * kLower, joined[((size_t)w * a.rows + r) * kJoinRow + tid], x);
                    den = fmaf(weight(ml.y, M), ml.z, den);
                }
                if (!whole) {
                    a.part_o[(slot * a.rows + r) * kD + tid] = x;
                    if (tid == 0) a.part_ml[slot * a.rows + r] = make_float4(R, M, den, any_bad ? 1.f : 0.f);
                } else if (!any_bad) {
                    a.o[((size_t)cb * a.heads_q + head0 + r) * kD + tid] = __float2bfloat16_rn(quotient(x, R, M, den));
                }
            }
        }
        // All four warps leave together when one of them has given up waiting.
        uint32_t stop;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.u32 q, %1, 0;\n\t"
            "bar.red.or.pred p, 1, %2, q;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(stop)
            : "r"(run && !aborted ? 0u : 1u), "n"(kComputeWarps * 32)
            : "memory");
        if (stop) {
            give_up(a.gave_up + blockIdx.x, aborted, produced, &issued_s, full(0), a.stages, a.fault,
                    a.part_ml + (size_t)blockIdx.x * 2 * a.rows, a.rows);
            return;
        }
        piece = 1;
    }
    if (tid == 0) a.gave_up[blockIdx.x] = 0;
}

// Joins the pieces of every row of blocks that more than one share holds.  One block per
// (sequence, key/value head, row tile); its warps share out the query heads and, with few of
// those, the pieces of a head (one long sequence has as many pieces as an eighth of the
// shares: read one after the other they took 17 us, by sixteen warps 11, both under the profiler
// with cold caches; with four or eight warps the call took 87 and 82 us against 69).
// A lane has four columns.
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const PagedArgs a)
{
    __shared__ int tmp[33];
    __shared__ int before_s;
    __shared__ float4 sums[kCombineWarps][32];
    pdl_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_seq = a.heads_kv * a.row_tiles;
    // What the shares report, by a block without a row of its own (beside a row's work it took 20 registers more: 70 us
    // against 67.5 for the e4m3 batch).
    if (blockIdx.x == gridDim.x - 1) {
        if (a.err)
            for (int c = tid; c < a.shares; c += kCombineThreads)
                if (const int where = a.gave_up[c]) latch_error(a.err, STREE_ERR_TIMEOUT, -1, where, c);
        return;
    }
    const int item = blockIdx.x % per_seq, b = blockIdx.x / per_seq;
    int n_all = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kCombineThreads) {
        int t;
        const int before = block_scan(b0 + tid < a.batch ? blocks_of(a, b0 + tid) : 0, tmp, &t);
        if (b0 + tid == b) before_s = n_all + before;
        n_all += t;
    }
    __syncthreads();
    const int nb = blocks_of(a, b);
    if (nb == 0) return;
    const long long total = (long long)n_all * per_seq;
    const long long begin = (long long)before_s * per_seq + (long long)item * nb, end = begin + nb;
    // The share that holds block x: the last c with share_begin(c) <= x.
    const int shares = (int)min((long long)a.shares, total);
    const int c0 = (int)(((begin + 1) * shares - 1) / total), pieces = (int)((end * shares - 1) / total) - c0 + 1;
    if (pieces == 1) return;
    const int first = share_begin(total, c0, shares) == begin ? 0 : 1;
    const int hkv = item / a.row_tiles, rt = item % a.row_tiles;
    const int heads = a.group <= 8 ? 8 : kMaxHeads;
    const int rows = min(heads, a.group - rt * heads);
    int slices = kCombineWarps / rows;         // warps of a head, at most one per piece
    slices = min(max(slices, 1), pieces);
    const int r = warp / slices, slice = warp % slices;
    const bool mine = r < rows;
    auto at = [&](int k) { return ((size_t)(c0 + k) * 2 + (k == 0 ? first : 0)) * a.rows + r; };
    float R = -INFINITY, M = -INFINITY, den = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    if (mine) {
        for (int k = lane; k < pieces; k += 32) {
            const float4 ml = a.part_ml[at(k)];
            R = fmaxf(R, ml.x);
            M = fmaxf(M, ml.y);
            bad |= ml.w != 0.f;
        }
        bad = __any_sync(0xffffffffu, bad);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, d));
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        }
#pragma unroll 4
        for (int k = slice; k < pieces; k += slices) {
            const float4 ml = a.part_ml[at(k)];
            const float4 v = reinterpret_cast<const float4 *>(a.part_o + at(k) * kD)[lane];
            const float f = weight(ml.x, R);
            x.x = fmaf(f, v.x, x.x);
            x.y = fmaf(f, v.y, x.y);
            x.z = fmaf(f, v.z, x.z);
            x.w = fmaf(f, v.w, x.w);
        }
        sums[warp][lane] = x;
    }
    __syncthreads();
    if (!mine || bad || slice != 0) return;
    for (int k = lane; k < pieces; k += 32) {
        const float4 ml = a.part_ml[at(k)];
        den = fmaf(weight(ml.y, M), ml.z, den);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
    for (int w = 1; w < slices; ++w) {
        const float4 v = sums[warp + w][lane];
        x.x += v.x;
        x.y += v.y;
        x.z += v.z;
        x.w += v.w;
    }
    const uint2 w = make_uint2(pack_bf16(quotient(x.x, R, M, den), quotient(x.y, R, M, den)),
                               pack_bf16(quotient(x.z, R, M, den), quotient(x.w, R, M, den)));
    reinterpret_cast<uint2 *>(a.o + ((size_t)b * a.heads_q + hkv * a.group + rt * heads + r) * kD)[lane] = w;
}

constexpr int kMaxDevices = 64;
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
        const auto set = [](auto *f) { return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerCta); };
        if ((e = set(paged_attention_kernel<false, 1>)) != cudaSuccess || (e = set(paged_attention_kernel<false, 2>)) != cudaSuccess ||
            (e = set(paged_attention_kernel<true, 1>)) != cudaSuccess || (e = set(paged_attention_kernel<true, 2>)) != cudaSuccess)
            return e;
        int n = 0;
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        g_sms[dev] = n > 0 ? n : 1;
    }
    *sms = g_sms[dev];
    return cudaSuccess;
}

bool heads_ok(int heads_q, int heads_kv) { return heads_q >= 1 && heads_kv >= 1 && heads_q % heads_kv == 0; }

size_t paged_ws(int shares, int rows) { return (size_t)shares * (2 * rows * (kD * sizeof(float) + sizeof(float4)) + sizeof(int)); }

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace stree

using namespace stree;

extern "C" stree_status stree_paged_attention_workspace_size(int heads_q, int heads_kv, int head_dim, size_t *bytes)
{
    if (!bytes) return STREE_ERR_INVALID_ARG;
    if (!heads_ok(heads_q, heads_kv) || head_dim != kD) return STREE_ERR_UNSUPPORTED;
    int sms = 0;
    if (prepare(&sms) != cudaSuccess) return STREE_ERR_CUDA;
    const int group = heads_q / heads_kv;
    *bytes = paged_ws(kCtasPerSm * sms, group < kMaxHeads ? group : kMaxHeads);
    return STREE_OK;
}

extern "C" stree_status stree_paged_attention(const void *q, const void *k_pages, const void *v_pages,
                                              const uint8_t *k_scales, const uint8_t *v_scales,
                                              const int32_t *page_table, const int32_t *seq_len, int batch,
                                              int heads_q, int heads_kv, int head_dim, int n_pages, int page_size,
                                              int max_pages, float scale, stree_dtype dtype, stree_dtype cache_dtype,
                                              void *o, void *workspace, size_t workspace_bytes, int32_t *err_out,
                                              void *stream)
{
    if (!heads_ok(heads_q, heads_kv) || dtype != STREE_BF16) return STREE_ERR_UNSUPPORTED;
    stree_status st = check_cache(k_pages, v_pages, k_scales, v_scales, page_table, batch, heads_kv, head_dim, n_pages,
                                  page_size, max_pages, cache_dtype);
    if (st != STREE_OK) return st;
    if (!(scale > 0.f)) return STREE_ERR_INVALID_ARG;
    if (batch == 0) return STREE_OK;
    if (!q || !seq_len || !o || !workspace) return STREE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(seq_len, 4) || !aligned(err_out, 4))
        return STREE_ERR_MISALIGNED;
    PagedArgs a{};
    a.group = heads_q / heads_kv;
    const int nt = a.group <= 8 ? 1 : 2;
    a.rows = a.group < 8 * nt ? a.group : 8 * nt;
    a.row_tiles = (a.group + 8 * nt - 1) / (8 * nt);
    const bool e4m3 = cache_dtype == STREE_E4M3;
    a.blk = block_positions(e4m3);
    const long long blocks = ((long long)max_pages * page_size + a.blk - 1) / a.blk;
    if (blocks * batch > 0x7fffffffLL || (long long)batch * heads_kv * a.row_tiles >= 0x7fffffffLL)
        return STREE_ERR_UNSUPPORTED;
    int sms = 0;
    if (prepare(&sms) != cudaSuccess) return STREE_ERR_CUDA;
    // As many shares as the SMs hold CTAs, and no more than there can be blocks.
    const long long most = blocks * batch * heads_kv * a.row_tiles;
    a.shares = (int)(most < (long long)kCtasPerSm * sms ? most : (long long)kCtasPerSm * sms);
    const size_t need = paged_ws(a.shares, a.rows);
    if (workspace_bytes < need) return STREE_ERR_INVALID_ARG;
    a.box_rows = 8;
    while (a.box_rows < 64 && page_size % (2 * a.box_rows) == 0) a.box_rows *= 2;
    const long long rows = (long long)n_pages * heads_kv * page_size;
    CUtensorMap m_k, m_v;
    if (!encode_rows(&m_k, k_pages, e4m3, rows, a.box_rows) || !encode_rows(&m_v, v_pages, e4m3, rows, a.box_rows))
        return STREE_ERR_CUDA;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.table = page_table;
    a.lens = seq_len;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float4 *>(a.part_o + (size_t)a.shares * 2 * a.rows * kD);
    a.gave_up = reinterpret_cast<int *>(a.part_ml + (size_t)a.shares * 2 * a.rows);
    a.err = err_out;
    a.batch = batch;
    a.heads_q = heads_q;
    a.heads_kv = heads_kv;
    a.n_pages = n_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.scale_log2 = scale * 1.4426950408889634f;
    const WaitHook hook = wait_hook();
    a.wait_ns = hook.limit_ns;
    a.fault = hook.fault;
    const int stage = e4m3 ? stage_layout<true>().bytes : stage_layout<false>().bytes;
    const int join = kComputeWarps * a.rows * kJoinRow * (int)sizeof(float), slack = 1024, fixed = 3072;
    a.stages = (kSmemPerCta - join - slack - fixed) / stage;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    const size_t smem = (size_t)a.stages * stage + join + slack;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const auto kernel = e4m3 ? (nt == 1 ? paged_attention_kernel<true, 1> : paged_attention_kernel<true, 2>)
                             : (nt == 1 ? paged_attention_kernel<false, 1> : paged_attention_kernel<false, 2>);
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)a.shares + 1), kThreads, smem, s, m_k, m_v, a);
    if (e != cudaSuccess) return STREE_ERR_CUDA;
    return launch_pdl(paged_combine_kernel, dim3((unsigned)(batch * heads_kv * a.row_tiles) + 1), kCombineThreads, 0, s, a) ==
                   cudaSuccess
               ? STREE_OK
               : STREE_ERR_CUDA;
}
