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
// the two halves of a register as two bfloat16 numbers. Scales and zero points are
// dealt per tile too, [row][group of the tile].
//
// A code becomes the number 16 + c, exact in bfloat16 with c in the upper
// four bits of its mantissa: one shift and one and-or for two weights, and no
// conversion. Adding -(16 + z) x, another product on the matrix instruction, into
// the same float32 accumulators leaves the group's sum of x (c - z). The terms are at
// most three times as large as x (c - z)'s own, so the sums lose less than two bits.
//
// Bound by HBM: N K / 2 bytes of codes for up to about a hundred rows of x.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kTileRows = 16, kTileCols = 128;

// where the parts of a packed weight lie
struct W4Layout {
    int64_t row_tiles, col_tiles;
    int64_t scales, zeros, bytes;  // offsets (the codes are at 0), total
};
__host__ __device__ inline W4Layout w4_layout(int64_t N, int64_t K, int G, DType scale_dtype, bool has_zeros)
{
    W4Layout l;
    l.row_tiles = (N + kTileRows - 1) / kTileRows;
    l.col_tiles = (K + kTileCols - 1) / kTileCols;
    l.scales = l.row_tiles * l.col_tiles * 1024;
    const int64_t n = l.row_tiles * l.col_tiles * (kTileRows * kTileCols / G);
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
    const int gpt = kTileCols / a.group;
    const int64_t n_scales = l.row_tiles * l.col_tiles * kTileRows * gpt;
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
        const int64_t tile = i / (kTileRows * gpt), n = tile / l.col_tiles * kTileRows + i / gpt % kTileRows;
        const int64_t g = tile % l.col_tiles * gpt + i % gpt;
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
            const int64_t at = (tile * kTileRows + lane % 16) * (kTileCols / a.group) + i * 32 / a.group;
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
// -(16 + z) twice, as bfloat16
__device__ __forceinline__ uint32_t w4_zero_pair(uint32_t z) { return z * 0x00080008u + 0xc180c180u; }

// What a lane reads of the scales or zero points of a tile: ROWS rows of GPT groups
template <int BYTES>
__device__ __forceinline__ void load_bytes(rsrc_t r, uint32_t off, uint32_t* w)
{
    if constexpr (BYTES == 1) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
    } else if constexpr (BYTES == 2) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    } else if constexpr (BYTES == 4) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
    } else if constexpr (BYTES == 8) {
        typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
        const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, off + i * 16, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i * 4 + j] = v[j];
        }
    }
}
template <typename TS>
__device__ __forceinline__ float scale_at(const uint32_t* w, int i)
{
    if constexpr (sizeof(TS) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}

constexpr uint32_t kNowhere = 0x40000000u;  // an offset beyond every buffer here: reads zero

// A workgroup takes NT row tiles of W and MT tiles of 16 rows of x; its wavefronts
// deal the column tiles among themselves in runs of DEPTH, whose loads all go out
// before the first is used, and their sums are joined in LDS in a fixed order.
// Tiles beyond the last read as zero codes with zero scales.
template <int MT, int NT, int DEPTH, int G, typename TS, bool ZEROS>
__global__ __launch_bounds__(512) void w4_gemm_kernel(W4GemmArgs a, W4Layout l)
{
    extern __shared__ f32x4 part[];  // [wavefront][NT * MT][lane]
    constexpr int STEPS = G / 32;    // matrix instructions per group
    constexpr int GPT = kTileCols / G;
    constexpr int SB = 4 * GPT * sizeof(TS);  // a lane's scales: the four rows of its results
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int col = lane % 16, quad = lane / 16;
    const int64_t nt0 = (int64_t)blockIdx.x * NT, m0 = (int64_t)blockIdx.y * (MT * 16);
    const int K = (int)a.K, col_tiles = (int)l.col_tiles;
    const rsrc_t xr = make_rsrc(static_cast<const bf16_t*>(a.x) + m0 * a.x_ld,
                                ((min(a.M - m0, (int64_t)MT * 16) - 1) * a.x_ld + a.K) * 2);
    rsrc_t wr[NT], sr[NT], zr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int64_t at = min(nt0 + n, l.row_tiles - 1) * l.col_tiles;
        wr[n] = make_rsrc(a.packed + at * 1024, l.col_tiles * 1024);
        sr[n] = make_rsrc(a.packed + l.scales + at * (16 * GPT * sizeof(TS)), l.col_tiles * (16 * GPT * sizeof(TS)));
        if constexpr (ZEROS) zr[n] = make_rsrc(a.packed + l.zeros + at * (16 * GPT), l.col_tiles * (16 * GPT));
    }
    uint32_t xoff[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        xoff[t] = m0 + t * 16 + col < a.M ? (uint32_t)(((t * 16 + col) * a.x_ld + quad * 8) * 2) : kNowhere;

    f32x4 tot[NT][MT] = {};
    for (int run = wave * DEPTH; run < col_tiles; run += waves * DEPTH) {
        u32x4_t c[DEPTH][NT];
        uint32_t sw[DEPTH][NT][SB / 4], zw[DEPTH][NT][GPT > 4 ? GPT / 4 : 1];
        bf16x8 xf[DEPTH][4][MT];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int kc = run + d;
#pragma unroll
            for (int n = 0; n < NT; ++n) c[d][n] = __builtin_amdgcn_raw_buffer_load_b128(wr[n], kc * 1024 + lane * 16, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                load_bytes<SB>(sr[n], kc * (SB * 4) + quad * SB, sw[d][n]);
                if constexpr (ZEROS) load_bytes<GPT>(zr[n], (kc * 16 + col) * GPT, zw[d][n]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = kc * kTileCols + i * 32;
                const uint32_t k2 = k < K ? (uint32_t)k * 2 : kNowhere;  // K is a multiple of 32
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    xf[d][i][t] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(xr, xoff[t] + k2, 0, 0));
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // (the compiler would put the loads of x off until they are used)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
            for (int g = 0; g < GPT; ++g)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4 acc[MT] = {};
                    const uint32_t zp = ZEROS ? w4_zero_pair((zw[d][n][0] >> (8 * g)) & 255u) : 0xc1c0c1c0u;
                    const u32x4_t z4 = {zp, zp, zp, zp};
                    const bf16x8 zf = __builtin_bit_cast(bf16x8, z4);
#pragma unroll
                    for (int i = g * STEPS; i < (g + 1) * STEPS; ++i) {
                        const bf16x8 wf = w4_operand(c[d][n][i]);
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[d][i][t], acc[t], 0, 0, 0);
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(zf, xf[d][i][t], acc[t], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float s = scale_at<TS>(sw[d][n], r * GPT + g);
#pragma unroll
                        for (int t = 0; t < MT; ++t) tot[n][t][r] = fmaf(s, acc[t][r], tot[n][t][r]);
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

template <int MT, int NT, int DEPTH, int G, typename TS, bool ZEROS>
hipError_t launch_gemm_tiles(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    const int64_t blocks = (l.row_tiles + NT - 1) / NT;
    int waves = 4;
    while (waves < 8 && blocks * waves < 4096) waves *= 2;
    const dim3 grid((unsigned)blocks, (unsigned)((a.M + MT * 16 - 1) / (MT * 16)));
    hipLaunchKernelGGL((w4_gemm_kernel<MT, NT, DEPTH, G, TS, ZEROS>), grid, dim3(waves * 64), waves * NT * MT * 1024, s, a, l);
    return hipGetLastError();
}

template <int G, typename TS, bool ZEROS>
hipError_t launch_gemm_form(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    if (a.M <= 16) return launch_gemm_tiles<1, 1, 4, G, TS, ZEROS>(a, l, s);
    if (a.M <= 32) return launch_gemm_tiles<2, 2, 2, G, TS, ZEROS>(a, l, s);
    return launch_gemm_tiles<4, 2, 1, G, TS, ZEROS>(a, l, s);
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
