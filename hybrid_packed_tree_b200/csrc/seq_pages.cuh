// seq_pages.cuh -- packed sequences and paged caches: finding a sequence's share of a
// flattened list of work, checking offsets and page tables, the 8-bit cache rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "stree_internal.cuh"
#include "tc_ptx.cuh"

namespace stree {

constexpr int kCacheDim = 128;                 // head dim of every cached row

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void pdl_start()
{
    launch_dependents();
    wait_dependency();
}

// One launch that may start while its predecessor on the stream drains (every
// kernel launched this way begins with pdl_start before it touches memory, or waits where it says).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

// The waits of a kernel's warp roles: bounded (about a second), and small, since a copy of the
// code stands at each of some twenty waits and several roles share the instruction cache.  A
// wait that runs out leaves its number in `aborted` (a shared int, zero before); every other
// wait of the CTA then gives up too, and when all roles have ended the kernel reports it.
__device__ __forceinline__ bool wait_one(volatile int *aborted, uint32_t bar, uint32_t parity, int where,
                                         uint32_t limit_ns = (uint32_t)ptx::kWaitLimitNs)
{
    if (ptx::mbar_try_wait(bar, parity & 1)) return true;
    const uint32_t t0 = ptx::globaltimer_lo();
#pragma unroll 1
    while (!ptx::mbar_try_wait(bar, parity & 1)) {
        if (*aborted) return false;
        if (ptx::globaltimer_lo() - t0 > limit_ns) {
            *aborted = where;
            return false;
        }
    }
    return true;
}

// All lanes of a warp wait together, with one answer.
__device__ __forceinline__ bool wait_warp(volatile int *aborted, uint32_t bar, uint32_t parity, int where,
                                          uint32_t limit_ns = (uint32_t)ptx::kWaitLimitNs)
{
    return __all_sync(0xffffffffu, wait_one(aborted, bar, parity, where, limit_ns));
}

// A sequence's packed rows [begin, end); an offset pair that is not ascending
// inside [0, total] gives an empty sequence.
__device__ __forceinline__ int2 seq_range(const int32_t *cu, int b, int total)
{
    const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
    return lo < 0 || hi < lo || hi > total ? make_int2(0, 0) : make_int2(lo, hi);
}

// Exclusive sum of `v` over the block's threads and the block's total.  `tmp`: 33
// ints of shared memory.  Every thread of the block calls it.
__device__ __forceinline__ int block_scan(int v, int *tmp, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const int w = lane < nw ? tmp[lane] : 0;
        int t = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += u;
        }
        __syncwarp();
        if (lane < nw) tmp[lane] = t - w;
        if (lane == 31) tmp[32] = t;
    }
    __syncthreads();
    *total = tmp[32];
    return tmp[warp] + s - v;
}

// Finds the sequence that holds element `x` of the list in which sequence b has
// count(b) elements: found[0] = b, found[1] = the elements before it (found[0] = -1
// when x lies past the end).  Returns the length of the list.  `found`: 2 ints and
// `tmp`: 33 ints of shared memory.  Every thread of the block calls it.
template <typename Count>
__device__ __forceinline__ int block_find(int batch, int x, Count count, int *tmp, int *found)
{
    if (threadIdx.x == 0) found[0] = -1;
    int base = 0;
    for (int b0 = 0; b0 < batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        const int n = b < batch ? count(b) : 0;
        int total;
        const int before = base + block_scan(n, tmp, &total);
        if (x >= before && x < before + n) {
            found[0] = b;
            found[1] = before;
        }
        base += total;
    }
    __syncthreads();
    return base;
}

// The error word of a call over packed sequences and page tables, written by one
// block of the grid that does nothing else: cleared, then the first sequence found
// whose offsets are not ascending inside [0, total], whose tokens do not fit its
// table, or one of whose used pages is out of range.  The other blocks take the
// same decisions for the rows they handle and skip them.
struct PageCheck {
    const int32_t *cu;        // [batch + 1], or NULL: `count` tokens are given per sequence
    const int32_t *count;     // [batch] (cu NULL)
    const int32_t *start;     // [batch] first position, or NULL (0)
    const int32_t *table;     // [batch, max_pages], or NULL: no pages
    int batch, total, n_pages, page_size, max_pages;
    int clamp;                // counts are clamped to [0, clamp] instead of refused (-1: refused)
};

__device__ inline void check_pages(const PageCheck &c, int32_t *err)
{
    if (!err) return;
    if (threadIdx.x < 4) err[threadIdx.x] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int b = warp; b < c.batch; b += nw) {
        int n;
        if (c.cu) {
            const int lo = __ldg(c.cu + b), hi = __ldg(c.cu + b + 1);
            if (lo < 0 || hi < lo || hi > c.total) {
                if (lane == 0) latch_error(err, STREE_ERR_BAD_SEQ, b, lo, hi);
                continue;
            }
            n = hi - lo;
        } else {
            n = __ldg(c.count + b);
            if (c.clamp >= 0) n = min(max(n, 0), c.clamp);
        }
        if (!c.table || n == 0) continue;
        const int at = c.start ? __ldg(c.start + b) : 0;
        if (n < 0 || at < 0 || (long long)at + n > (long long)c.max_pages * c.page_size) {
            if (lane == 0) latch_error(err, STREE_ERR_BAD_PAGE, b, at, n);
            continue;
        }
        for (int p = at / c.page_size + lane; p <= (at + n - 1) / c.page_size; p += 32) {
            const int id = __ldg(c.table + (size_t)b * c.max_pages + p);
            if (id < 0 || id >= c.n_pages) latch_error(err, STREE_ERR_BAD_PAGE, b, p, id);
        }
    }
}

// ---------------------------------------------------------------- 8-bit cache rows

// A row of 128 values is held as e4m3 under one scale 2^(s - 127), s one byte: the
// least power of two that brings the row's largest finite magnitude to 448 or below,
// s within [9, 246].  A power of two costs e4m3 no precision (its step is relative)
// and makes the scaling and the reading back exact: every value read back is a bf16.
__device__ __forceinline__ uint32_t scale_of_top(uint32_t top_bits)
{
    const int e = (int)(top_bits >> 7), m = (int)(top_bits & 127);
    return (uint32_t)min(max(e - 8 + (m > 96 ? 1 : 0), 9), 246);   // 448 = 1.75 2^8: mantissa 96 / 128
}

// Largest magnitude bits of two packed bf16, infinities and NaN left out.
__device__ __forceinline__ uint32_t finite_top2(uint32_t w)
{
    const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
    return max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u);
}

__device__ __forceinline__ float power_of_two(uint32_t biased) { return __uint_as_float(biased << 23); }

// Two bf16 times a power of two -> two e4m3 (nearest even, beyond 448 to 448, NaN kept).
__device__ __forceinline__ uint32_t quantise2(uint32_t w, float inv)
{
    const float lo = __uint_as_float(w << 16) * inv, hi = __uint_as_float(w & 0xffff0000u) * inv;
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 -> two fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

// Four e4m3 -> two pairs of fp16, exactly.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Two e4m3 times a power of two -> two bf16, exactly (a scale within [9, 246]).
__device__ __forceinline__ uint32_t dequantise2(uint32_t w, float scale)
{
    const uint32_t h = e4m3x2_to_f16x2(w);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    return *reinterpret_cast<const uint32_t *>(&r);
}

}  // namespace stree
