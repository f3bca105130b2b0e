// kda_norm.hip -- residual addition + RMSNorm in front of a block's projections,
// also with a norm of the block's output before it is added, its output in
// float32, bfloat16 or block FP8 (gfx950).
//
// Per row: h = x + residual, residual_out = round(h), and
//   y = h / sqrt(mean(h^2) + eps) * w,
// or, for the W8A8 projections, y quantized in groups of 128 columns: scale =
// max|y| / 448, code = E4M3(y / scale) (the format of kda_quantize_fp8, whose
// own pass over the row this saves).
//
// Everything is formed from the float32 h (not from the rounded residual_out),
// and rounded once when stored: rounding h before the norm would put the
// residual's storage error into y a second time.
//
// Bound by HBM: one pass, the row held in registers between the sum of squares
// and the normalisation. A lane owns 8 consecutive columns per step (16-byte
// accesses for bfloat16, two of them for float32), so a group of 128 columns
// is 16 neighbouring lanes of one wavefront and its maximum a 16-lane
// reduction.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

struct Fp8Out {};  // output type tag: E4M3 codes + scales

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f)
{
    if constexpr (sizeof(T) == 2) {
        Vec16<bf16_t>::unpack(ld16(p), f);
    } else {
        Vec16<float>::unpack(ld16(p), f);
        Vec16<float>::unpack(ld16(p + 4), f + 4);
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f)
{
    if constexpr (sizeof(T) == 2) {
        st16(p, Vec16<bf16_t>::pack(f));
    } else {
        st16(p, Vec16<float>::pack(f));
        st16(p + 4, Vec16<float>::pack(f + 4));
    }
}

// Sum over the TPR threads of one row (64: a wavefront; more: the workgroup).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part)
{
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += part[i];
    }
    return v;
}

// 8 normalised values of columns c .. c + 7 of row m -> memory
template <typename TY, typename Args>
__device__ __forceinline__ void emit8(const Args& a, int64_t m, int64_t c, const float* y)
{
    if constexpr (!__is_same(TY, Fp8Out)) {
        store8(static_cast<TY*>(a.y) + m * a.y_ld + c, y);
    } else {
        // the maximum of |y| over the group's 16 lanes, taken on the bit
        // patterns: ordered like the magnitudes, with NaN above infinity, so a
        // NaN is kept
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
#pragma unroll
        for (int s = 8; s >= 1; s >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s, 64));
        float scale = __uint_as_float(top) / 448.0f;
        if (!(scale > 0.0f)) scale = 1.0f;  // an all-zero group (or a NaN, which the codes then show)
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = y[i] / scale;
            q[i] = v > 448.0f ? 448.0f : (v < -448.0f ? -448.0f : v);  // keeps NaN
        }
        uint2 w;
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], p, true);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
        w.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], p, true);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + m * a.y_ld + c) = w;
        if ((threadIdx.x & 15) == 0) a.scales[m * a.scale_ld + c / 128] = scale;
    }
}

// TPR threads per row, each NV steps of 8 columns (TPR * 8 * NV >= K).
template <typename TX, typename TR, typename TY, bool RES, int TPR, int NV>
__global__ __launch_bounds__(256) void add_norm_kernel(AddNormArgs a)
{
    __shared__ float part[4];
    const int t = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    if (m >= a.M) return;  // whole wavefronts (TPR = 64) leave; TPR = 256 has one row a workgroup
    const TX* x = static_cast<const TX*>(a.x) + m * a.x_ld;
    float h[NV][8], r[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = (int64_t)(v * TPR + t) * 8;
        if (c < a.K) {
            load8(x + c, h[v]);
            if constexpr (RES) load8(static_cast<const TR*>(a.res) + m * a.res_ld + c, r[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = (int64_t)(v * TPR + t) * 8;
        if (c >= a.K) continue;
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] += r[v][i];
            if (a.res_out) store8(static_cast<TR*>(a.res_out) + m * a.res_out_ld + c, h[v]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += h[v][i] * h[v][i];
    }
    const float rn = 1.0f / sqrtf(row_sum<TPR>(ss, part) / (float)a.K + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = (int64_t)(v * TPR + t) * 8;
        if (c >= a.K) continue;  // K is a multiple of 128 for FP8: whole 16-lane groups leave
        float y[8], w[8];
        load8(a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[v][i] * rn * w[i];
        emit8<TY>(a, m, c, y);
    }
}

// Rows too wide for the registers: the row is read again (from the caches) for
// the second half. 2048 rows of 16,384 (bfloat16) 73 us, with E4M3 output 70 us (one
// read of everything at a copy's rate: 53 and 47).
template <typename TX, typename TR, typename TY, bool RES>
__global__ __launch_bounds__(256) void add_norm_wide_kernel(AddNormArgs a)
{
    __shared__ float part[4];
    const int64_t m = blockIdx.x;
    const TX* x = static_cast<const TX*>(a.x) + m * a.x_ld;
    auto row8 = [&](int64_t c, float* h) {
        load8(x + c, h);
        if constexpr (RES) {
            float r[8];
            load8(static_cast<const TR*>(a.res) + m * a.res_ld + c, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += r[i];
        }
    };
    float ss = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < a.K; c += 2048) {
        float h[8];
        row8(c, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += h[i] * h[i];
    }
    const float rn = 1.0f / sqrtf(row_sum<256>(ss, part) / (float)a.K + a.eps);
    for (int64_t c = threadIdx.x * 8; c < a.K; c += 2048) {
        float h[8], w[8];
        row8(c, h);  // before this thread's own store: residual_out may be residual
        if constexpr (RES)
            if (a.res_out) store8(static_cast<TR*>(a.res_out) + m * a.res_out_ld + c, h);
        load8(a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * rn * w[i];
        emit8<TY>(a, m, c, h);
    }
}

template <typename TX, typename TR, typename TY, bool RES>
hipError_t launch_rows(const AddNormArgs& a, hipStream_t s)
{
    const dim3 block(256), rows((unsigned)a.M);
    if (a.K <= 1024)
        hipLaunchKernelGGL((add_norm_kernel<TX, TR, TY, RES, 64, 2>), dim3((unsigned)((a.M + 3) / 4)), block, 0, s, a);
    else if (a.K <= 4096)
        hipLaunchKernelGGL((add_norm_kernel<TX, TR, TY, RES, 256, 2>), rows, block, 0, s, a);
    else if (a.K <= 8192)
        hipLaunchKernelGGL((add_norm_kernel<TX, TR, TY, RES, 256, 4>), rows, block, 0, s, a);
    else
        hipLaunchKernelGGL((add_norm_wide_kernel<TX, TR, TY, RES>), rows, block, 0, s, a);
    return hipGetLastError();
}

template <typename TX, typename TY>
hipError_t launch_res(const AddNormArgs& a, hipStream_t s)
{
    if (!a.res) return launch_rows<TX, TX, TY, false>(a, s);
    return a.res_dtype == F32 ? launch_rows<TX, float, TY, true>(a, s) : launch_rows<TX, bf16_t, TY, true>(a, s);
}

template <typename TX>
hipError_t launch_out(const AddNormArgs& a, hipStream_t s)
{
    if (a.scales) return launch_res<TX, Fp8Out>(a, s);
    return a.y_dtype == F32 ? launch_res<TX, float>(a, s) : launch_res<TX, bf16_t>(a, s);
}

// ---------------------------------------------------------------- a norm after the block, too
//   h = residual_scale residual + branch_scale act(gate) x / sqrt(mean(x^2) + post_eps) w_post
//   residual_out = round(h),  y = h / sqrt(mean(h^2) + eps) w
// One pass as above, with two sums over the row; the row, its residual and gate are in
// registers before the first (all loads go out together). Everything is float32 until stored.
enum Gate : int { kNoGate = 0, kGate = 1, kSigmoid = 2 };

// the 8 columns of h from those of x (normalised by rn), residual r and gate g
template <int GATE>
__device__ __forceinline__ void combine8(const SandwichArgs& a, int64_t c, float rn, const float* r, const float* g, float* h)
{
    float w[8];
    load8(a.w_post + c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float n = h[i] * rn * w[i];
        if constexpr (GATE == kGate) n *= g[i];
        if constexpr (GATE == kSigmoid) n *= sigmoidf_(g[i]);
        h[i] = fmaf(a.branch_scale, n, a.residual_scale * r[i]);
    }
}

template <typename TX, typename TR, typename TG, typename TY, int GATE, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void sandwich_kernel(SandwichArgs a)
{
    constexpr int THREADS = TPR > 256 ? TPR : 256;
    __shared__ float part[2][TPR / 64];
    const int t = threadIdx.x % TPR;
    const int64_t m = a.row0 + (int64_t)blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR;
    if (m >= a.M) return;  // whole wavefronts (TPR = 64) leave; otherwise a workgroup has one row
    const TX* x = static_cast<const TX*>(a.x) + m * a.x_ld;
    float h[NV][8], r[NV][8], g[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = (int64_t)(v * TPR + t) * 8;
        if (c < a.K) {
            load8(x + c, h[v]);
            load8(static_cast<const TR*>(a.res) + m * a.res_ld + c, r[v]);
            if constexpr (GATE != kNoGate) load8(static_cast<const TG*>(a.gate) + m * a.gate_ld + c, g[v]);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if ((int64_t)(v * TPR + t) * 8 < a.K)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += h[v][i] * h[v][i];
    const float rx = 1.0f / sqrtf(row_sum<TPR>(ss, part[0]) / (float)a.K + a.post_eps);
    ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = (int64_t)(v * TPR + t) * 8;
        if (c >= a.K) continue;
        combine8<GATE>(a, c, rx, r[v], g[v], h[v]);
        if (a.res_out) store8(static_cast<TR*>(a.res_out) + m * a.res_out_ld + c, h[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += h[v][i] * h[v][i];
    }
    const float rh = 1.0f / sqrtf(row_sum<TPR>(ss, part[1]) / (float)a.K + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t c = (int64_t)(v * TPR + t) * 8;
        if (c >= a.K) continue;  // K is a multiple of 128 for FP8: whole 16-lane groups leave
        float y[8], w[8];
        load8(a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[v][i] * rh * w[i];
        emit8<TY>(a, m, c, y);
    }
}

// Rows too wide for the registers: x is read again for h, and h formed again (from the
// caches) for y. residual_out is written in the last sweep.
template <typename TX, typename TR, typename TG, typename TY, int GATE>
__global__ __launch_bounds__(1024) void sandwich_wide_kernel(SandwichArgs a)
{
    __shared__ float part[2][16];
    const int64_t m = a.row0 + blockIdx.x;
    const TX* x = static_cast<const TX*>(a.x) + m * a.x_ld;
    float ss = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < a.K; c += 8192) {
        float h[8];
        load8(x + c, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += h[i] * h[i];
    }
    const float rx = 1.0f / sqrtf(row_sum<1024>(ss, part[0]) / (float)a.K + a.post_eps);
    auto row8 = [&](int64_t c, float* h) {
        float r[8], g[8];
        load8(x + c, h);
        load8(static_cast<const TR*>(a.res) + m * a.res_ld + c, r);
        if constexpr (GATE != kNoGate) load8(static_cast<const TG*>(a.gate) + m * a.gate_ld + c, g);
        combine8<GATE>(a, c, rx, r, g, h);
    };
    ss = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < a.K; c += 8192) {
        float h[8];
        row8(c, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += h[i] * h[i];
    }
    const float rh = 1.0f / sqrtf(row_sum<1024>(ss, part[1]) / (float)a.K + a.eps);
    for (int64_t c = threadIdx.x * 8; c < a.K; c += 8192) {
        float h[8], w[8];
        row8(c, h);  // before this thread's own store: residual_out may be residual
        if (a.res_out) store8(static_cast<TR*>(a.res_out) + m * a.res_out_ld + c, h);
        load8(a.w + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * rh * w[i];
        emit8<TY>(a, m, c, h);
    }
}

// launch(args, grid) for all rows, ROWS to a workgroup of THREADS. A launch holds less than
// 2^32 threads, which rows of 512 and more pass below the row limit: calls that large go
// out in several launches, each from its row0 on.
template <int ROWS, int THREADS, typename Launch>
hipError_t in_row_ranges(SandwichArgs a, Launch launch)
{
    constexpr int64_t MOST = ((int64_t)1 << 31) / THREADS * ROWS;
    for (a.row0 = 0; a.row0 < a.M; a.row0 += MOST) {
        launch(a, dim3((unsigned)((min(a.M - a.row0, MOST) + ROWS - 1) / ROWS)));
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Few columns a thread, so that many rows are under way at once: us with THREADS x NV, rows of
// bfloat16 (a gate of their own) 8191 x 4096 65.6 with 512 x 1, 68.0 with 256 x 2; 2000 x 8192
// 38.3 with 512 x 2, 41.1 with 256 x 4; 2048 x 16,384 without a gate 55.9 with 1024 x 2, 79.9
// read again; 1000 x 30,720 75 with 1024 x 4, 90 read again (a copy's rate: 65.5, 32.0, 52.4, 60.0).
template <typename TX, typename TR, typename TG, typename TY, int GATE, int TPR, int NV>
hipError_t sandwich_launch(const SandwichArgs& a, hipStream_t s)
{
    constexpr int THREADS = TPR > 256 ? TPR : 256;
    return in_row_ranges<THREADS / TPR, THREADS>(a, [s](const SandwichArgs& part, dim3 grid) {
        hipLaunchKernelGGL((sandwich_kernel<TX, TR, TG, TY, GATE, TPR, NV>), grid, dim3(THREADS), 0, s, part);
    });
}

template <typename TX, typename TR, typename TG, typename TY, int GATE>
hipError_t sandwich_rows(const SandwichArgs& a, hipStream_t s)
{
    if (a.K <= 1024) return sandwich_launch<TX, TR, TG, TY, GATE, 64, 2>(a, s);
    if (a.K <= 2048) return sandwich_launch<TX, TR, TG, TY, GATE, 256, 1>(a, s);
    if (a.K <= 4096) return sandwich_launch<TX, TR, TG, TY, GATE, 512, 1>(a, s);
    if (a.K <= 8192) return sandwich_launch<TX, TR, TG, TY, GATE, 512, 2>(a, s);
    if (a.K <= 16384) return sandwich_launch<TX, TR, TG, TY, GATE, 1024, 2>(a, s);
    if (a.K <= 32768) return sandwich_launch<TX, TR, TG, TY, GATE, 1024, 4>(a, s);
    return in_row_ranges<1, 1024>(a, [s](const SandwichArgs& part, dim3 grid) {
        hipLaunchKernelGGL((sandwich_wide_kernel<TX, TR, TG, TY, GATE>), grid, dim3(1024), 0, s, part);
    });
}

template <typename TX, typename TR, typename TY>
hipError_t sandwich_gate(const SandwichArgs& a, hipStream_t s)
{
    if (!a.gate) return sandwich_rows<TX, TR, float, TY, kNoGate>(a, s);
    if (a.gate_dtype == F32)
        return a.sigmoid ? sandwich_rows<TX, TR, float, TY, kSigmoid>(a, s) : sandwich_rows<TX, TR, float, TY, kGate>(a, s);
    return a.sigmoid ? sandwich_rows<TX, TR, bf16_t, TY, kSigmoid>(a, s) : sandwich_rows<TX, TR, bf16_t, TY, kGate>(a, s);
}

template <typename TX, typename TR>
hipError_t sandwich_out(const SandwichArgs& a, hipStream_t s)
{
    if (a.scales) return sandwich_gate<TX, TR, Fp8Out>(a, s);
    return a.y_dtype == F32 ? sandwich_gate<TX, TR, float>(a, s) : sandwich_gate<TX, TR, bf16_t>(a, s);
}

template <typename TX>
hipError_t sandwich_res(const SandwichArgs& a, hipStream_t s)
{
    return a.res_dtype == F32 ? sandwich_out<TX, float>(a, s) : sandwich_out<TX, bf16_t>(a, s);
}

}  // namespace

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t s)
{
    if (a.M == 0) return hipSuccess;
    return a.x_dtype == F32 ? launch_out<float>(a, s) : launch_out<bf16_t>(a, s);
}

hipError_t launch_sandwich(const SandwichArgs& a, hipStream_t s)
{
    if (a.M == 0) return hipSuccess;
    return a.x_dtype == F32 ? sandwich_res<float>(a, s) : sandwich_res<bf16_t>(a, s);
}

}  // namespace kda
