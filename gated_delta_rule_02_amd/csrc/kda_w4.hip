// kda_w4.hip -- products with 4-bit weights and group scales (gfx950).
//
//   y[m, n] = sum_k x[m, k] W[n, k] (+ residual),  W[n, k] = s[n, k/G] (c[n, k] - z[n, k/G])
//
// with codes c in 0..15, one scale and zero point (8 if there are none) per row
// and group of G = 32, 64 or 128 columns; x bfloat16, float32 accumulation.
//
// Packed layout (w4_pack_kernel, once per weight): tiles of 16 rows x 128 columns,
// 1 KiB each, a row of tiles after the other; in a tile lane l holds 16 bytes,
// row l % 16; its 32-bit word i is the eight codes of columns 32 i + 8 (l / 16) + j,
// which is lane l's operand of a 16x16x32 matrix instruction. So a wavefront's
// load is one contiguous KiB whatever G is. The codes of an even j sit in nibble
// j / 2, of an odd one in nibble 4 + j / 2: shifted and masked, each pair falls into
// the two halves of a register as two bfloat16 numbers.
//
// A code becomes the number 16 + c, exact in bfloat16 with c in the upper
// four bits of its mantissa: one shift and one and-or for two weights, and no
// conversion. The group's sum is then put right in float32,
//   sum_k x (c - z) = sum_k x (16 + c) - (16 + z) sum_k x,
// with sum_k x from the same instruction with ones in place of the weights, in
// the layout of the accumulator. The terms are at most three times as large as
// x (c - z)'s own, so the float32 sums lose less than two bits to it.
//
// Bound by HBM: N K / 2 bytes of codes for up to about a hundred rows of x.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kTileRows = 16, kTileCols = 128;

// where the parts of a packed weight lie
struct W4Layout {
    int64_t row_tiles, col_tiles, groups;  // groups of one row, the padding's included
    int64_t scales, zeros, bytes;          // offsets (the codes are at 0), total
};
__host__ __device__ inline W4Layout w4_layout(int64_t N, int64_t K, int G, DType scale_dtype, bool has_zeros)
{
    W4Layout l;
    l.row_tiles = (N + kTileRows - 1) / kTileRows;
    l.col_tiles = (K + kTileCols - 1) / kTileCols;
    l.groups = l.col_tiles * (kTileCols / G);
    l.scales = l.row_tiles * l.col_tiles * 1024;
    const int64_t n = l.row_tiles * l.groups * kTileRows;
    l.zeros = l.scales + n * (scale_dtype == F32 ? 4 : 2);
    l.bytes = has_zeros ? l.zeros + n : l.zeros;
    return l;
}

// bfloat16 pairs 16 + c from a packed word: operand register p of 4
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int p)
{
    const uint32_t t = p == 0 ? w << 3 : w >> (4 * p - 3);
    return (t & 0x00780078u) | 0x41804180u;
}
__device__ __forceinline__ bf16x8 w4_operand(uint32_t w)
{
    const u32x4_t r = {w4_pair(w, 0), w4_pair(w, 1), w4_pair(w, 2), w4_pair(w, 3)};
    return __builtin_bit_cast(bf16x8, r);
}

// ---------------------------------------------------------------- packing
__global__ __launch_bounds__(256) void w4_pack_kernel(W4PackArgs a, W4Layout l)
{
    const int64_t words = l.row_tiles * l.col_tiles * 256;
    const int64_t n_scales = l.row_tiles * l.groups * kTileRows;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
        const int step = i & 3, lane = (i >> 2) & 63;
        const int64_t tile = i >> 8, n = tile / l.col_tiles * kTileRows + lane % 16;
        const int64_t k = tile % l.col_tiles * kTileCols + step * 32 + lane / 16 * 8;
        uint32_t w = 0;
        if (n < a.N && k < a.K) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(a.codes + n * a.codes_ld + k / 2);
#pragma unroll
            for (int j = 0; j < 8; ++j) w |= ((c >> (4 * j)) & 15u) << (4 * (j % 2 * 4 + j / 2));
        }
        reinterpret_cast<uint32_t*>(a.packed)[i] = w;
    }
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_scales; i += (int64_t)gridDim.x * 256) {
        const int64_t tg = i / kTileRows, n = tg / l.groups * kTileRows + i % kTileRows, g = tg % l.groups;
        const bool in = n < a.N && g < a.K / a.group;
        if (a.scale_dtype == F32)
            reinterpret_cast<float*>(a.packed + l.scales)[i] = in ? static_cast<const float*>(a.scales)[n * a.scales_ld + g] : 0.0f;
        else
            reinterpret_cast<bf16_t*>(a.packed + l.scales)[i] = in ? static_cast<const bf16_t*>(a.scales)[n * a.scales_ld + g] : bf16_t(0);
        if (a.zeros) a.packed[l.zeros + i] = in ? (a.zeros[n * a.zeros_ld + g] & 15) : 0;
    }
}

// ---------------------------------------------------------------- expansion
// A wavefront per tile: W in bfloat16, for products of many rows.
template <typename TS, bool ZEROS>
__global__ __launch_bounds__(256) void w4_expand_kernel(W4ExpandArgs a, W4Layout l)
{
    const int lane = threadIdx.x & 63;
    const int64_t tiles = l.row_tiles * l.col_tiles;
    for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += (int64_t)gridDim.x * 4) {
        const int64_t nt = tile / l.col_tiles, kc = tile % l.col_tiles, n = nt * kTileRows + lane % 16;
        const u32x4_t c = ld16(a.packed + (tile * 64 + lane) * 16);
        if (n >= a.N) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = kc * kTileCols + i * 32 + lane / 16 * 8;
            if (k >= a.K) break;
            const int64_t at = (nt * l.groups + k / a.group) * kTileRows + lane % 16;
            const float s = ld(reinterpret_cast<const TS*>(a.packed + l.scales) + at);
            const float z = ZEROS ? (float)a.packed[l.zeros + at] : 8.0f;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = ((float)((c[i] >> (4 * (j % 2 * 4 + j / 2))) & 15u) - z) * s;
            st16(a.out + n * a.out_ld + k, Vec16<bf16_t>::pack(w));
        }
    }
}

// ---------------------------------------------------------------- product
// A workgroup takes NT row tiles of W and MT tiles of 16 rows of x; its
// wavefronts deal the column tiles among themselves and their sums are joined in
// LDS in a fixed order.
template <int MT, int NT, int G, typename TS, bool ZEROS>
__global__ __launch_bounds__(512) void w4_gemm_kernel(W4GemmArgs a, W4Layout l)
{
    extern __shared__ f32x4 part[];  // [wavefront][NT * MT][lane]
    constexpr int STEPS = G / 32;    // matrix instructions per group
    constexpr int GPT = kTileCols / G;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int col = lane % 16, quad = lane / 16;
    const int64_t nt0 = (int64_t)blockIdx.x * NT, m0 = (int64_t)blockIdx.y * (MT * 16);
    const uint8_t* w = a.packed + lane * 16;
    const rsrc_t xr = make_rsrc(static_cast<const bf16_t*>(a.x) + m0 * a.x_ld,
                                ((min(a.M - m0, (int64_t)MT * 16) - 1) * a.x_ld + a.K) * 2);
    uint32_t xoff[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        xoff[t] = m0 + t * 16 + col < a.M ? (uint32_t)(((t * 16 + col) * a.x_ld + quad * 8) * 2) : 0x80000000u;
    const u32x4_t one4 = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, one4);

    f32x4 tot[NT][MT] = {};
    for (int64_t kc = wave; kc < l.col_tiles; kc += waves) {
        u32x4_t c[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t nt = min(nt0 + n, l.row_tiles - 1);
            c[n] = ld16(w + (nt * l.col_tiles + kc) * 1024);
        }
#pragma unroll
        for (int g = 0; g < GPT; ++g) {
            f32x4 acc[NT][MT] = {}, xs[MT] = {};
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
                const int i = g * STEPS + st;
                const uint32_t k2 = (uint32_t)(kc * kTileCols + i * 32) * 2;
                const bool in = kc * kTileCols + i * 32 < a.K;  // K is a multiple of 32
                bf16x8 xf[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    // rows and columns that are not there: an offset beyond the buffer reads zero
                    xf[t] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(xr, in ? xoff[t] + k2 : 0x80000000u, 0, 0));
                    xs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xf[t], xs[t], 0, 0, 0);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const bf16x8 wf = w4_operand(c[n][i]);
#pragma unroll
                    for (int t = 0; t < MT; ++t) acc[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[t], acc[n][t], 0, 0, 0);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int64_t nt = min(nt0 + n, l.row_tiles - 1);
                const int64_t at = (nt * l.groups + kc * GPT + g) * kTileRows + quad * 4;
                const f32x4 s = ld4(reinterpret_cast<const TS*>(a.packed + l.scales) + at);
                uint32_t z4 = 0;
                if constexpr (ZEROS) z4 = *reinterpret_cast<const uint32_t*>(a.packed + l.zeros + at);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float z = ZEROS ? -16.0f - (float)((z4 >> (8 * r)) & 255u) : -24.0f;
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        tot[n][t][r] = fmaf(s[r], fmaf(z, xs[t][r], acc[n][t][r]), tot[n][t][r]);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[(wave * (NT * MT) + n * MT + t) * 64 + lane] = tot[n][t];
    __syncthreads();
    for (int i = wave; i < NT * MT; i += waves) {
        f32x4 v = part[i * 64 + lane];
        for (int j = 1; j < waves; ++j) {
            const f32x4 o = part[(j * (NT * MT) + i) * 64 + lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += o[r];
        }
        const int64_t n = (nt0 + i / MT) * kTileRows + quad * 4, m = m0 + i % MT * 16 + col;
        if (m >= a.M) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (n + r >= a.N) break;
            float f = v[r];
            if (a.res) f += a.res_dtype == F32 ? static_cast<const float*>(a.res)[m * a.res_ld + n + r]
                                               : bf16_to_f32(static_cast<const bf16_t*>(a.res)[m * a.res_ld + n + r]);
            if (a.y_dtype == F32) static_cast<float*>(a.y)[m * a.y_ld + n + r] = f;
            else static_cast<bf16_t*>(a.y)[m * a.y_ld + n + r] = f32_to_bf16(f);
        }
    }
}

template <int MT, int NT, int G, typename TS, bool ZEROS>
hipError_t launch_gemm_tiles(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    const int64_t blocks = (l.row_tiles + NT - 1) / NT;
    int waves = 4;
    while (waves < 8 && blocks * waves < 4096) waves *= 2;
    const dim3 grid((unsigned)blocks, (unsigned)((a.M + MT * 16 - 1) / (MT * 16)));
    hipLaunchKernelGGL((w4_gemm_kernel<MT, NT, G, TS, ZEROS>), grid, dim3(waves * 64), waves * NT * MT * 1024, s, a, l);
    return hipGetLastError();
}

template <int G, typename TS, bool ZEROS>
hipError_t launch_gemm_form(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    if (a.M <= 16) return launch_gemm_tiles<1, 1, G, TS, ZEROS>(a, l, s);
    if (a.M <= 32) return launch_gemm_tiles<2, 2, G, TS, ZEROS>(a, l, s);
    return launch_gemm_tiles<4, 2, G, TS, ZEROS>(a, l, s);
}

template <typename TS, bool ZEROS>
hipError_t launch_gemm_group(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    if (a.group == 32) return launch_gemm_form<32, TS, ZEROS>(a, l, s);
    if (a.group == 64) return launch_gemm_form<64, TS, ZEROS>(a, l, s);
    return launch_gemm_form<128, TS, ZEROS>(a, l, s);
}

}  // namespace

size_t w4_packed_bytes(int64_t N, int64_t K, int group, DType scale_dtype, bool has_zeros)
{
    return (size_t)w4_layout(N, K, group, scale_dtype, has_zeros).bytes;
}

hipError_t launch_w4_pack(const W4PackArgs& a, hipStream_t s)
{
    const W4Layout l = w4_layout(a.N, a.K, a.group, a.scale_dtype, a.zeros != nullptr);
    const int64_t blocks = min(l.row_tiles * l.col_tiles, (int64_t)8192);
    hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, l);
    return hipGetLastError();
}

hipError_t launch_w4_expand(const W4ExpandArgs& a, hipStream_t s)
{
    const W4Layout l = w4_layout(a.N, a.K, a.group, a.scale_dtype, a.has_zeros);
    const dim3 grid((unsigned)min((l.row_tiles * l.col_tiles + 3) / 4, (int64_t)1 << 20)), block(256);
    if (a.scale_dtype == F32) {
        if (a.has_zeros) hipLaunchKernelGGL((w4_expand_kernel<float, true>), grid, block, 0, s, a, l);
        else hipLaunchKernelGGL((w4_expand_kernel<float, false>), grid, block, 0, s, a, l);
    } else {
        if (a.has_zeros) hipLaunchKernelGGL((w4_expand_kernel<bf16_t, true>), grid, block, 0, s, a, l);
        else hipLaunchKernelGGL((w4_expand_kernel<bf16_t, false>), grid, block, 0, s, a, l);
    }
    return hipGetLastError();
}

hipError_t launch_w4_gemm(const W4GemmArgs& a, hipStream_t s)
{
    const W4Layout l = w4_layout(a.N, a.K, a.group, a.scale_dtype, a.has_zeros);
    if (a.scale_dtype == F32)
        return a.has_zeros ? launch_gemm_group<float, true>(a, l, s) : launch_gemm_group<float, false>(a, l, s);
    return a.has_zeros ? launch_gemm_group<bf16_t, true>(a, l, s) : launch_gemm_group<bf16_t, false>(a, l, s);
}

}  // namespace kda
