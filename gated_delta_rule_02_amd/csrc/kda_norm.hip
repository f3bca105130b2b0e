// kda_norm.hip -- residual addition + RMSNorm in front of a block's projections,
// its output in float32, bfloat16 or block FP8 (gfx950).
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

// Sum over the threads of one row (TPR = 64: a wavefront; 256: the workgroup).
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
template <typename TY>
__device__ __forceinline__ void emit8(const AddNormArgs& a, int64_t m, int64_t c, const float* y)
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

}  // namespace

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t s)
{
    if (a.M == 0) return hipSuccess;
    return a.x_dtype == F32 ? launch_out<float>(a, s) : launch_out<bf16_t>(a, s);
}

}  // namespace kda
