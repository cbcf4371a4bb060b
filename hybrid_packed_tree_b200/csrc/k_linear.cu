// k_linear.cu -- linear attention with a decay for each head (gated linear attention,
// and with alpha = exp(dt A), beta = dt the selective SSM of Mamba2): the single-token
// step, the prompt pass on CUDA cores, and the entry points, sm_100a.
//
// Per sequence and value head h (query/key head g = h / (Hv / Hk)):
//   S_t = alpha_t S_{t-1} + beta_t v_t k_t^T,   o_t = S_t q_t + D_h v_t.
//
// Both kernels hold rows of S ([dv, dk], fp32) in registers: a warp has eight rows,
// a lane four columns of each (columns 4 l .. 4 l + 3, and 128 further where dk is
// above 128), so the update is one multiply and one fused multiply-add per element
// and the eight row products with q are reduced over the lanes by one butterfly that
// halves the rows at each step (nine shuffles for eight sums).
//
// The step reads and writes the whole state once and is bound by HBM: every load of a
// warp's rows (eight independent 16-byte loads per lane) is issued before any use, and the
// loads are marked as streaming, so that the lines read leave L2 before the lines written
// (64 sequences of 32 heads of 128 x 128: 42 us, 6.4 TB/s; 53 us with plain loads; a
// streaming mark on the stores changes nothing).
// The prompt pass walks a sequence token by token with the tokens staged in shared
// memory sixteen at a time, the next tile's loads in flight meanwhile; it serves fp32 inputs
// and the shapes that the tensor-core kernel (k_linear_tc.cu) does not take, and its time is
// the walk's latency (35 us at 96 tokens before the tiles were double-buffered and two tokens
// taken together, so that one's sums over the lanes run beside the other's update).
#include "linear.cuh"
#include "seq_pages.cuh"

namespace stree {
namespace {

constexpr int kRows = 8;                       // state rows per warp
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kFewWarps = 256;                 // prompt: below so many warps of eight rows, two rows a warp

// Sums of eight values over the warp: lane l returns the total of value (l >> 2) & 7.
__device__ __forceinline__ float reduce8(const float (&p)[8], int lane)
{
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {              // bit 4 of the lane picks the upper half of the rows
        const bool up = lane & 16;
        const float keep = up ? p[i + 4] : p[i], give = up ? p[i] : p[i + 4];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        const float keep = up ? a[i + 2] : a[i], give = up ? a[i] : a[i + 2];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
    }
    const bool up = lane & 4;
    const float keep = up ? b[1] : b[0], give = up ? b[0] : b[1];
    float c = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    c += __shfl_xor_sync(0xffffffffu, c, 2);
    c += __shfl_xor_sync(0xffffffffu, c, 1);
    return c;
}

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// CH: 128-column parts of a row (dk up to 128 CH; lanes past dk hold zeros).
template <typename T, int CH>
__global__ void __launch_bounds__(kThreads) linear_step_kernel(const LinearArgs a)
{
    pdl_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = a.dv / kRows;
    const long long item = (long long)blockIdx.x * kWarps + warp;
    if (item >= (long long)a.batch * a.heads_v * groups) return;
    const long long bh = item / groups;
    const int r0 = (int)(item % groups) * kRows;
    const int b = (int)(bh / a.heads_v), h = (int)(bh % a.heads_v), g = h / (a.heads_v / a.heads_k);
    const size_t srow = ((size_t)bh * a.dv + r0) * a.dk;
    const T *q = static_cast<const T *>(a.q) + ((size_t)b * a.heads_k + g) * a.dk;
    const T *k = static_cast<const T *>(a.k) + ((size_t)b * a.heads_k + g) * a.dk;
    const T *v = static_cast<const T *>(a.v) + (size_t)bh * a.dv + r0;
    float4 S[CH][kRows], qv[CH], kv[CH];
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = c * 128 + lane * 4;
        const bool in = col < a.dk;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            S[c][r] = in ? __ldcs(reinterpret_cast<const float4 *>(a.S0 + srow + (size_t)r * a.dk + col)) : zero;
        qv[c] = in ? load4(q + col) : zero;
        kv[c] = in ? load4(k + col) : zero;
    }
    const float alpha = __ldg(a.alpha + bh), beta = a.beta ? __ldg(a.beta + bh) : 1.f;
    float p[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const float w = beta * load1(v + r);
        p[r] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float4 &s = S[c][r];
            s.x = fmaf(w, kv[c].x, alpha * s.x);
            s.y = fmaf(w, kv[c].y, alpha * s.y);
            s.z = fmaf(w, kv[c].z, alpha * s.z);
            s.w = fmaf(w, kv[c].w, alpha * s.w);
            const int col = c * 128 + lane * 4;
            if (col < a.dk) *reinterpret_cast<float4 *>(a.S_new + srow + (size_t)r * a.dk + col) = s;
            p[r] = fmaf(s.x, qv[c].x, fmaf(s.y, qv[c].y, fmaf(s.z, qv[c].z, fmaf(s.w, qv[c].w, p[r]))));
        }
    }
    const float o = reduce8(p, lane);
    const int r = lane >> 2;
    if ((lane & 3) == 0)
        store1(static_cast<T *>(a.o) + (size_t)bh * a.dv + r0 + r, a.skip ? fmaf(__ldg(a.skip + h), load1(v + r), o) : o);
}

// Sums of R values over the warp (R = 8 or 2): lane l returns the total of value l / (32 / R).
template <int R>
__device__ __forceinline__ float reduce_rows(const float (&p)[R], int lane)
{
    if constexpr (R == 8) {
        return reduce8(p, lane);
    } else {
        const bool up = lane & 16;
        float c = (up ? p[1] : p[0]) + __shfl_xor_sync(0xffffffffu, up ? p[0] : p[1], 16);
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
        return c;
    }
}

// R: state rows per warp.
template <typename T, int CH, int R>
__global__ void __launch_bounds__(kThreads) linear_prompt_kernel(const LinearArgs a)
{
    constexpr int kTile = 16 / CH;             // tokens staged at a time
    constexpr int kSlice = kWarps * R;         // rows of the CTA
    constexpr int kPart = kTile * CH * 32 / kThreads, kPartV = (kTile * kSlice + kThreads - 1) / kThreads;
    __shared__ float4 qs[2][kTile][CH * 32], ks[2][kTile][CH * 32];
    __shared__ float vs[2][kTile][kSlice], al[2][kTile], be[2][kTile];
    pdl_start();
    if (blockIdx.x == gridDim.x - 1) {         // the error word
        PageCheck c{};
        c.cu = a.cu;
        c.batch = a.batch;
        c.total = a.total;
        check_pages(c, a.err);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slices = (a.dv + kSlice - 1) / kSlice;
    const int sl = blockIdx.x % slices;
    const long long bh = blockIdx.x / slices;
    const int b = (int)(bh / a.heads_v), h = (int)(bh % a.heads_v), g = h / (a.heads_v / a.heads_k);
    const int2 seq = seq_range(a.cu, b, a.total);
    const int c0 = sl * kSlice, r0 = c0 + warp * R;
    const bool rows = r0 < a.dv;               // dv is a multiple of eight: a warp's rows all exist or none does
    const size_t srow = ((size_t)bh * a.dv + r0) * a.dk;
    float2 S[CH][R][2];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int col = c * 128 + lane * 4;
            const float4 x = rows && a.S0 && col < a.dk ? load4(a.S0 + srow + (size_t)r * a.dk + col) : make_float4(0.f, 0.f, 0.f, 0.f);
            S[c][r][0] = make_float2(x.x, x.y);
            S[c][r][1] = make_float2(x.z, x.w);
        }
    const float skip = a.skip ? __ldg(a.skip + h) : 0.f;
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    // A tile of tokens travels global -> registers (in flight while the one before is worked on) -> shared.
    float4 pq[kPart], pk[kPart];
    float pv[kPartV], pa = 1.f, pb = 1.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
            const int e = i * kThreads + tid, t = t0 + e / (CH * 32), col = e % (CH * 32) * 4;
            const bool in = t < seq.y && col < a.dk;
            const size_t at = ((size_t)t * a.heads_k + g) * a.dk + col;
            pq[i] = in ? load4(q + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            pk[i] = in ? load4(k + at) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kPartV; ++i) {
            const int e = i * kThreads + tid, t = t0 + e / kSlice, col = c0 + e % kSlice;
            pv[i] = e < kTile * kSlice && t < seq.y && col < a.dv ? load1(v + ((size_t)t * a.heads_v + h) * a.dv + col) : 0.f;
        }
        if (tid < kTile && t0 + tid < seq.y) {
            pa = __ldg(a.alpha + (size_t)(t0 + tid) * a.heads_v + h);
            pb = a.beta ? __ldg(a.beta + (size_t)(t0 + tid) * a.heads_v + h) : 1.f;
        }
    };
    auto token = [&](int z, int t) {
        const float alpha = al[z][t], beta = be[z][t];
        float p[R];
        float2 kv[CH][2], qv[CH][2];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float4 x = ks[z][t][c * 32 + lane], y = qs[z][t][c * 32 + lane];
            kv[c][0] = make_float2(x.x, x.y);
            kv[c][1] = make_float2(x.z, x.w);
            qv[c][0] = make_float2(y.x, y.y);
            qv[c][1] = make_float2(y.z, y.w);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float w = beta * vs[z][t][warp * R + r];
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float2 &s = S[c][r][e];
                    s = ptx::ffma2(make_float2(w, w), kv[c][e], ptx::fmul2(make_float2(alpha, alpha), s));
                    sum = ptx::ffma2(s, qv[c][e], sum);
                }
            p[r] = sum.x + sum.y;
        }
        return reduce_rows<R>(p, lane);
    };
    fetch(seq.x);
    int z = 0;
    for (int t0 = seq.x; t0 < seq.y; t0 += kTile, z ^= 1) {
        const int n = min(kTile, seq.y - t0);
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
            const int e = i * kThreads + tid;
            qs[z][e / (CH * 32)][e % (CH * 32)] = pq[i];
            ks[z][e / (CH * 32)][e % (CH * 32)] = pk[i];
        }
#pragma unroll
        for (int i = 0; i < kPartV; ++i) {
            const int e = i * kThreads + tid;
            if (e < kTile * kSlice) vs[z][e / kSlice][e % kSlice] = pv[i];
        }
        if (tid < kTile) {
            al[z][tid] = pa;
            be[z][tid] = pb;
        }
        __syncthreads();                       // one a tile: the other buffer was read before the last one
        if (t0 + kTile < seq.y) fetch(t0 + kTile);
        if (!rows) continue;
        T *out = static_cast<T *>(a.o) + ((size_t)t0 * a.heads_v + h) * a.dv + r0 + lane / (32 / R);
        const bool writes = lane % (32 / R) == 0;
        auto put = [&](int t, float o) {
            if (writes) store1(out + (size_t)t * a.heads_v * a.dv, fmaf(skip, vs[z][t][warp * R + lane / (32 / R)], o));
        };
        int t = 0;
        for (; t + 2 <= n; t += 2) {           // two tokens: the second's update beside the first's sums
            const float o0 = token(z, t), o1 = token(z, t + 1);
            put(t, o0);
            put(t + 1, o1);
        }
        if (t < n) put(t, token(z, t));
    }
    if (!a.S_new || !rows) return;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int col = c * 128 + lane * 4;
            if (col < a.dk)
                *reinterpret_cast<float4 *>(a.S_new + srow + (size_t)r * a.dk + col) =
                    make_float4(S[c][r][0].x, S[c][r][0].y, S[c][r][1].x, S[c][r][1].y);
        }
}

template <typename T>
cudaError_t launch_step(const LinearArgs &a, cudaStream_t s)
{
    const long long items = (long long)a.batch * a.heads_v * (a.dv / kRows);
    const dim3 grid((unsigned)((items + kWarps - 1) / kWarps));
    return a.dk <= 128 ? launch_pdl(linear_step_kernel<T, 1>, grid, kThreads, 0, s, a)
                       : launch_pdl(linear_step_kernel<T, 2>, grid, kThreads, 0, s, a);
}

template <typename T, int R>
cudaError_t launch_prompt_rows(const LinearArgs &a, cudaStream_t s)
{
    const int slices = (a.dv + kWarps * R - 1) / (kWarps * R);
    const dim3 grid((unsigned)((long long)a.batch * a.heads_v * slices + 1));
    return a.dk <= 128 ? launch_pdl(linear_prompt_kernel<T, 1, R>, grid, kThreads, 0, s, a)
                       : launch_pdl(linear_prompt_kernel<T, 2, R>, grid, kThreads, 0, s, a);
}

// Eight rows a warp spend the fewest instructions on a token, two the least time: with few
// rows in all the walk's latency counts (fp32; sequences of 96 and 33 tokens, 8 heads of 32 x 64,
// 64 warps of eight rows: 15.3 us with two rows, 19.9 with eight; 256 tokens, 80 heads of 64 x
// 128, 640 warps: 100 and 95; four such sequences: 279 and 161).
template <typename T>
cudaError_t launch_prompt(const LinearArgs &a, cudaStream_t s)
{
    const long long warps = (long long)a.batch * a.heads_v * (a.dv / kRows);
    return warps <= kFewWarps ? launch_prompt_rows<T, 2>(a, s) : launch_prompt_rows<T, 8>(a, s);
}

bool shape_ok(int batch, int heads_v, int heads_k, int dk, int dv, stree_dtype dtype)
{
    return batch >= 0 && heads_v >= 1 && heads_k >= 1 && heads_v % heads_k == 0 && dk >= 8 && dk <= kMaxDim &&
           dk % 8 == 0 && dv >= 8 && dv <= kMaxDim && dv % 8 == 0 && (dtype == STREE_F32 || dtype == STREE_BF16) &&
           (long long)batch * heads_v * dv <= 0x7fffffffLL;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// S_new may be S0 itself (each row is read before it is written, by the same lanes),
// and no other output may overlap an input.
stree_status check_linear(const LinearArgs &a)
{
    const bool rows = !a.cu || a.total > 0;    // no packed row: no row pointer is used
    if (rows && (!a.q || !a.k || !a.v || !a.alpha || !a.o)) return STREE_ERR_INVALID_ARG;
    const void *ptrs[] = {a.q, a.k, a.v, a.S0, a.o, a.S_new};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return STREE_ERR_MISALIGNED;
    if (!aligned(a.alpha, 4) || !aligned(a.beta, 4) || !aligned(a.skip, 4) || !aligned(a.cu, 4) || !aligned(a.err, 4))
        return STREE_ERR_MISALIGNED;
    return STREE_OK;
}

LinearArgs make_args(const void *q, const void *k, const void *v, const float *alpha, const float *beta,
                     const float *skip, const float *S0, int batch, int heads_v, int heads_k, int dk, int dv,
                     stree_dtype dtype, void *o, float *S_new)
{
    LinearArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.alpha = alpha;
    a.beta = beta;
    a.skip = skip;
    a.S0 = S0;
    a.batch = batch;
    a.heads_v = heads_v;
    a.heads_k = heads_k;
    a.dk = dk;
    a.dv = dv;
    a.dtype = dtype;
    a.o = o;
    a.S_new = S_new;
    return a;
}

}  // namespace
}  // namespace stree

using namespace stree;

extern "C" stree_status stree_linear_step(const void *q, const void *k, const void *v, const float *alpha,
                                          const float *beta, const float *skip, const float *S0, int batch,
                                          int heads_v, int heads_k, int dk, int dv, stree_dtype dtype, void *o,
                                          float *S_new, void *stream)
{
    if (!shape_ok(batch, heads_v, heads_k, dk, dv, dtype)) return STREE_ERR_UNSUPPORTED;
    if (batch == 0) return STREE_OK;
    const LinearArgs a = make_args(q, k, v, alpha, beta, skip, S0, batch, heads_v, heads_k, dk, dv, dtype, o, S_new);
    if (!S0 || !S_new) return STREE_ERR_INVALID_ARG;
    const stree_status st = check_linear(a);
    if (st != STREE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == STREE_BF16 ? launch_step<__nv_bfloat16>(a, s) : launch_step<float>(a, s);
    return e == cudaSuccess ? STREE_OK : STREE_ERR_CUDA;
}

extern "C" stree_status stree_linear_prompt_workspace_size(int batch, int total, int heads_v, int heads_k, int dk,
                                                           int dv, stree_dtype dtype, size_t *bytes)
{
    if (!bytes) return STREE_ERR_INVALID_ARG;
    if (!shape_ok(batch, heads_v, heads_k, dk, dv, dtype) || total < 0) return STREE_ERR_UNSUPPORTED;
    *bytes = 0;
    if (batch == 0 || !linear_tc_supported(heads_v, heads_k, dk, dv, dtype)) return STREE_OK;
    return linear_tc_workspace(batch, total, heads_v, dv, bytes) == cudaSuccess ? STREE_OK : STREE_ERR_CUDA;
}

extern "C" stree_status stree_linear_prompt(const void *q, const void *k, const void *v, const float *alpha,
                                            const float *beta, const float *skip, const float *S0,
                                            const int32_t *cu_seqlens, int total, int batch, int heads_v, int heads_k,
                                            int dk, int dv, stree_dtype dtype, void *o, float *S_new, void *workspace,
                                            size_t workspace_bytes, int32_t *err_out, void *stream)
{
    if (!shape_ok(batch, heads_v, heads_k, dk, dv, dtype) || total < 0) return STREE_ERR_UNSUPPORTED;
    if (batch == 0) return STREE_OK;
    LinearArgs a = make_args(q, k, v, alpha, beta, skip, S0, batch, heads_v, heads_k, dk, dv, dtype, o, S_new);
    a.cu = cu_seqlens;
    a.total = total;
    a.err = err_out;
    if (!cu_seqlens) return STREE_ERR_INVALID_ARG;
    const stree_status st = check_linear(a);
    if (st != STREE_OK) return st;
    if (workspace && !aligned(workspace, 16)) return STREE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (linear_tc_supported(heads_v, heads_k, dk, dv, dtype))
        return launch_linear_tc(a, workspace, workspace_bytes, s) == cudaSuccess ? STREE_OK : STREE_ERR_CUDA;
    const cudaError_t e = dtype == STREE_BF16 ? launch_prompt<__nv_bfloat16>(a, s) : launch_prompt<float>(a, s);
    return e == cudaSuccess ? STREE_OK : STREE_ERR_CUDA;
}
