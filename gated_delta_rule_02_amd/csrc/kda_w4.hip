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
// the same float32 accumulators leaves the group's sum of x (c - z). What is summed is up to
// 31 |x| whatever c - z is, so an output is off by a part of sum |s| |x| (32 + c + z), not of its
// own size: for uniform codes by 1.2e-7 (norm of all, 41,024 x 4096), for codes within 1 of the
// zero point by 2e-7 to 6e-7, and codes at it throughout need not give exactly 0.
//
// Bound by HBM (N K / 2 bytes of codes) for one row: 41,024 x 4096 in 20 us, 4.3 TB/s. For
// more, by the instructions of a column tile, since those of the vector unit find little room
// beside the matrix instruction's with two wavefronts a SIMD: 64 rows 30 to 36 us (30 with
// part of the weights in the last-level cache), where each of a wavefront's turns takes 64
// matrix and about 170 vector instructions, and the weights at a copy's rate 18 us.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

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

// bfloat16 pairs 16 + c from a packed word. The two constants are in registers, and the
// compiler kept from knowing them: it would take an and and an or with a constant each
// in place of one and-or.
struct W4Unpack {
    uint32_t mask, bias;
    __device__ __forceinline__ W4Unpack()
    {
        asm("s_mov_b32 %0, 0x00780078" : "=s"(mask));
        asm("v_mov_b32 %0, 0x41804180" : "=v"(bias));
    }
    __device__ __forceinline__ bf16x8 operator()(uint32_t w) const
    {
        const u32x4_t r = {((w << 3) & mask) | bias, ((w >> 1) & mask) | bias, ((w >> 5) & mask) | bias, ((w >> 9) & mask) | bias};
        return __builtin_bit_cast(bf16x8, r);
    }
};

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
// A wavefront per tile: W in bfloat16, for products of many rows. 41,024 x 4096 98 us, 4.3 TB/s.
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

// BYTES of a lane's scales or zero points of a tile
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

// v + residual -> columns n .. n + 3 of row m of y
__device__ __forceinline__ void store4(const W4GemmArgs& a, int64_t m, int64_t n, f32x4 v)
{
    if (m >= a.M) return;
    if (n + 4 <= a.N && (a.y_ld | a.res_ld) % 4 == 0) {  // (res_ld is 0 without a residual)
        if (a.res) {
            const f32x4 r = a.res_dtype == F32 ? ld4(static_cast<const float*>(a.res) + m * a.res_ld + n)
                                               : ld4(static_cast<const bf16_t*>(a.res) + m * a.res_ld + n);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += r[i];
        }
        if (a.y_dtype == F32) st4(static_cast<float*>(a.y) + m * a.y_ld + n, v);
        else st4(static_cast<bf16_t*>(a.y) + m * a.y_ld + n, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= a.N) break;
        float f = v[i];
        if (a.res) f += a.res_dtype == F32 ? static_cast<const float*>(a.res)[m * a.res_ld + n + i]
                                           : bf16_to_f32(static_cast<const bf16_t*>(a.res)[m * a.res_ld + n + i]);
        if (a.y_dtype == F32) static_cast<float*>(a.y)[m * a.y_ld + n + i] = f;
        else static_cast<bf16_t*>(a.y)[m * a.y_ld + n + i] = f32_to_bf16(f);
    }
}

// A workgroup takes a row tile of W and 16 rows of x; its wavefronts deal the column
// tiles among themselves in runs of DEPTH, whose loads all go out before the first is
// used, and their sums are joined in LDS in a fixed order. Tiles beyond the last read
// as zero codes with zero scales.
template <int DEPTH, int G, typename TS, bool ZEROS>
__global__ __launch_bounds__(512) void w4_gemm_kernel(W4GemmArgs a, W4Layout l)
{
    extern __shared__ f32x4 part[];  // [wavefront][lane]
    constexpr int STEPS = G / 32;    // matrix instructions per group
    constexpr int GPT = kTileCols / G;
    constexpr int SB = 4 * GPT * sizeof(TS);  // a lane's scales: the four rows of its results
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int col = lane % 16, quad = lane / 16;
    const int64_t nt = blockIdx.x, m0 = (int64_t)blockIdx.y * 16, at = nt * l.col_tiles;
    const int K = (int)a.K, col_tiles = (int)l.col_tiles;
    const rsrc_t xr = make_rsrc(static_cast<const bf16_t*>(a.x) + m0 * a.x_ld, ((min(a.M - m0, (int64_t)16) - 1) * a.x_ld + a.K) * 2);
    const rsrc_t wr = make_rsrc(a.packed + at * 1024, l.col_tiles * 1024);
    const rsrc_t sr = make_rsrc(a.packed + l.scales + at * (16 * GPT * sizeof(TS)), l.col_tiles * (16 * GPT * sizeof(TS)));
    const rsrc_t zr = make_rsrc(a.packed + l.zeros + at * (16 * GPT), ZEROS ? l.col_tiles * (16 * GPT) : 0);
    const uint32_t xoff = m0 + col < a.M ? (uint32_t)((col * a.x_ld + quad * 8) * 2) : kNowhere;

    const W4Unpack unpack;
    f32x4 tot = {};
    for (int run = wave * DEPTH; run < col_tiles; run += waves * DEPTH) {
        u32x4_t c[DEPTH];
        uint32_t sw[DEPTH][SB / 4], zw[DEPTH][1];
        bf16x8 xf[DEPTH][4];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int kc = run + d;
            c[d] = __builtin_amdgcn_raw_buffer_load_b128(wr, kc * 1024 + lane * 16, 0, 0);
            load_bytes<SB>(sr, kc * (SB * 4) + quad * SB, sw[d]);
            if constexpr (ZEROS) load_bytes<GPT>(zr, (kc * 16 + col) * GPT, zw[d]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = kc * kTileCols + i * 32;
                const uint32_t k2 = k < K ? (uint32_t)k * 2 : kNowhere;  // K is a multiple of 32
                xf[d][i] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(xr, xoff + k2, 0, 0));
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // (the compiler would put the loads of x off until they are used)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
            for (int g = 0; g < GPT; ++g) {
                f32x4 acc = {};
                const uint32_t zp = ZEROS ? w4_zero_pair((zw[d][0] >> (8 * g)) & 255u) : 0xc1c0c1c0u;
                const u32x4_t z4 = {zp, zp, zp, zp};
                const bf16x8 zf = __builtin_bit_cast(bf16x8, z4);
#pragma unroll
                for (int i = g * STEPS; i < (g + 1) * STEPS; ++i) {
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(unpack(c[d][i]), xf[d][i], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(zf, xf[d][i], acc, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) tot[r] = fmaf(scale_at<TS>(sw[d], r * GPT + g), acc[r], tot[r]);
            }
    }
    part[wave * 64 + lane] = tot;
    __syncthreads();
    if (wave > 0) return;
    for (int j = 1; j < waves; ++j) {
        const f32x4 o = part[j * 64 + lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) tot[r] += o[r];
    }
    store4(a, m0 + col, nt * kTileRows + quad * 4, tot);
}

// More rows of x: what a compute unit takes in of x counts as much as the weights.
// 8 / KW wavefronts with NT row tiles of W each share the x of a column tile in LDS,
// copied there in whole lines; KW such groups take turns at the column tiles (four
// instead of two where row tiles are few: 64 x 4096 x 8192 14.7 us instead of 17.5).
// Copies and weights run two turns ahead. A group's sum of -24 x is formed once for the
// NT tiles and their products start from it; with zero points the sum of x is, and
// they are applied to it in float32.
template <int KW, int MT, int NT, int G, typename TS, bool ZEROS>
__global__ __launch_bounds__(512) void w4_rows_kernel(W4GemmArgs a, W4Layout l)
{
    constexpr int RW = 8 / KW, S = 3, kStage = MT * 4096;
    constexpr int CP = MT * 4 / RW;  // copies of a wavefront per column tile
    constexpr int STEPS = G / 32, GPT = kTileCols / G, SB = 4 * GPT * sizeof(TS), ZB = 4 * GPT;
    // loads of a wavefront per column tile
    constexpr int kLoads = CP + NT * (1 + (SB + 15) / 16 + (ZEROS ? 1 : 0));
    static_assert((KW - 1) * RW * NT * MT * 1024 <= KW * S * kStage, "the partial sums fit the stages");
    static_assert(kLoads < 64, "loads the wait can count");
    __shared__ __attribute__((aligned(16))) uint8_t smem[KW * S * kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % RW, kg = wave / RW, col = lane % 16, quad = lane / 16;
    const int64_t nt0 = ((int64_t)blockIdx.x * RW + rw) * NT, m0 = (int64_t)blockIdx.y * (MT * 16);
    const int K = (int)a.K, turns = ((int)l.col_tiles + KW - 1) / KW;
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
    // A copy takes 8 rows of x and 64 columns, whole cache lines (16 rows of 32, an operand, would
    // take in halves of twice as many); lane l row l / 8, and of its eight 16-byte pieces the one
    // whose number, xored with the row's, is l % 8, so that an operand's reads meet all banks. Four
    // copies a tile of rows: two columns of two.
    uint32_t xoff[CP];
#pragma unroll
    for (int p = 0; p < CP; ++p) {
        const int f = rw * CP + p, row = f / 4 * 16 + f % 4 / 2 * 8 + lane / 8;
        xoff[p] = m0 + row < a.M ? (uint32_t)(row * a.x_ld * 2) : kNowhere;
    }
    const int xcol = ((lane ^ (lane / 8)) & 7) * 8;
    const uint32_t xread = col / 8 * 2048 + col % 8 * 128 + ((quad ^ col) & 7) * 16;  // step 0; an odd one's: ^ 64
    uint8_t* ring = smem + kg * (S * kStage);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)ring;

    u32x4_t c[S][NT];
    uint32_t sw[S][NT][SB / 4], zw[S][NT][ZB / 4];
    // part p of CP + NT of a column tile's loads
    auto load = [&](int turn, int st, int p) {
        const int kc = turn * KW + kg;
        if (p < CP) {
            const int k = kc * kTileCols + (rw * CP + p) % 2 * 64 + xcol;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_void*)(uintptr_t)(lds0 + st * kStage + (rw * CP + p) * 1024), 16,
                                                     (int)(xoff[p] + (k < K ? (uint32_t)k * 2 : kNowhere)), 0, 0, 0);
        } else {
            const int n = p - CP;
            c[st][n] = __builtin_amdgcn_raw_buffer_load_b128(wr[n], kc * 1024 + lane * 16, 0, 0);
            load_bytes<SB>(sr[n], kc * (SB * 4) + quad * SB, sw[st][n]);
            if constexpr (ZEROS) load_bytes<ZB>(zr[n], kc * (ZB * 4) + quad * ZB, zw[st][n]);
        }
    };
    constexpr uint32_t kShift = ZEROS ? 0x3f803f80u : 0xc1c0c1c0u;  // 1, or -24
    const u32x4_t shift4 = {kShift, kShift, kShift, kShift};
    const bf16x8 shift = __builtin_bit_cast(bf16x8, shift4);

    f32x4 tot[NT][MT] = {};
#pragma unroll
    for (int p = 0; p < CP + NT; ++p) load(0, 0, p);
#pragma unroll
    for (int p = 0; p < CP + NT; ++p) load(1, 1, p);
    // (so that the compiler has nothing left of these to wait for within the loop)
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    const W4Unpack unpack;
    auto step = [&](int turn, int st, bool last) {
        // this turn's copies have landed (those of the next may be under way)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (last) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        else __builtin_amdgcn_s_waitcnt(0x0f70 | (kLoads & 15) | ((kLoads >> 4) << 14));
        lds_barrier();  // everyone's; and every read of the stage refilled now is done
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t* lds = ring + st * kStage;
#pragma unroll
        for (int g = 0; g < GPT; ++g) {
            bf16x8 xf[STEPS][MT];
            f32x4 xs[MT] = {};
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    xf[i][t] = __builtin_bit_cast(
                        bf16x8, ld16(lds + t * 4096 + (g * STEPS + i) / 2 * 1024 + (xread ^ ((g * STEPS + i) % 2 * 64))));
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int t = 0; t < MT; ++t) xs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(shift, xf[i][t], xs[t], 0, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f32x4 acc[MT] = {};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const bf16x8 wf = unpack(c[st][n][g * STEPS + i]);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[i][t], !ZEROS && i == 0 ? xs[t] : acc[t], 0, 0, 0);
                    // The loads of the turn after the next, spread over this one's products: issued in
                    // one go they hold a wavefront up for as long as its products take. (Beyond the last
                    // column tile too, where they read nothing: loads on a condition would make
                    // the compiler wait for all of them before it uses any.)
                    const int done = (g * NT + n) * STEPS + i;
#pragma unroll
                    for (int p = done * (CP + NT) / (4 * NT); p < (done + 1) * (CP + NT) / (4 * NT); ++p) {
                        if (last) break;
                        load(turn + 2, (st + 2) % S, p);
                        __builtin_amdgcn_sched_barrier(0x38f);  // (what is no memory access may cross)
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = r * GPT + g;
                    const float s = scale_at<TS>(sw[st][n], at);
                    const float z = ZEROS ? -16.0f - (float)((zw[st][n][at / 4] >> (8 * (at % 4))) & 255u) : 0.0f;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        if constexpr (ZEROS) tot[n][t][r] = fmaf(s, fmaf(z, xs[t][r], acc[t][r]), tot[n][t][r]);
                        else tot[n][t][r] = fmaf(s, acc[t][r], tot[n][t][r]);
                    }
                }
            }
        }
    };
    int turn = 0;
    for (; turn + S <= turns; turn += S) {
        step(turn, 0, false);
        step(turn + 1, 1, false);
        step(turn + 2, 2, false);
    }
    if (turn < turns) step(turn, 0, true);  // (turn + 1 is loaded, and nothing is left to load)
    if (turn + 1 < turns) step(turn + 1, 1, true);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the copies beyond the last column tile
    lds_barrier();                        // every wavefront has read its last stage
    f32x4* part = reinterpret_cast<f32x4*>(smem) + rw * (NT * MT * 64) + lane;  // of group 1, the others behind
    if (kg > 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < MT; ++t) part[((kg - 1) * RW * NT * MT + n * MT + t) * 64] = tot[n][t];
    }
    lds_barrier();
    if (kg > 0) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int q = 1; q < KW; ++q) {
                const f32x4 o = part[((q - 1) * RW * NT * MT + n * MT + t) * 64];
#pragma unroll
                for (int r = 0; r < 4; ++r) tot[n][t][r] += o[r];
            }
            store4(a, m0 + t * 16 + col, (nt0 + n) * kTileRows + quad * 4, tot[n][t]);
        }
}

template <int DEPTH, int G, typename TS, bool ZEROS>
hipError_t launch_gemm_tiles(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    const int waves = (int)min((l.col_tiles + DEPTH - 1) / DEPTH, (int64_t)8);
    const dim3 grid((unsigned)l.row_tiles, (unsigned)((a.M + 15) / 16));
    hipLaunchKernelGGL((w4_gemm_kernel<DEPTH, G, TS, ZEROS>), grid, dim3(waves * 64), waves * 1024, s, a, l);
    return hipGetLastError();
}

template <int KW, int MT, int NT, int G, typename TS, bool ZEROS>
hipError_t launch_gemm_rows(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    constexpr int TILES = 8 / KW * NT;
    const dim3 grid((unsigned)((l.row_tiles + TILES - 1) / TILES), (unsigned)((a.M + MT * 16 - 1) / (MT * 16)));
    hipLaunchKernelGGL((w4_rows_kernel<KW, MT, NT, G, TS, ZEROS>), grid, dim3(512), 0, s, a, l);
    return hipGetLastError();
}

// The form: the least of `start + rounds (tile + steps step)` us, with rounds of workgroups
// over the 256 compute units and steps of a tile, column tiles (w4_gemm_kernel: a part of
// a step follows the rows of x that there are) or turns at KW of them; a part follows the bytes
// of scales of a row of W in a column tile, and its zero points. The first form, which keeps
// nothing in LDS, unless another is 5 per cent better. Fitted to every form's time at 190 sizes (M
// 1..800, N 500..41,024, K 64..8,192, all groups and types): off by 7 to 12 per cent, and the form
// picked on average 1 per cent above the best of up to eleven that were tried (up to 16 rows; from
// 65 on 2.5), 38 at most. Always the first: 8 per cent up to 16 rows, 25 up to 64, 91 beyond, and at
// worst 5.3 times.
struct W4Form {
    int rows, row_tiles;  // of x and of W, per workgroup
    int turns;            // column tiles that a workgroup takes at a time, 0: one
    int least, most;      // rows of x: below, a smaller form does the same; above, a larger one nearly always better
    float start, tile, step, step_rows, step_scales, step_zeros;
    float cost(const W4GemmArgs& a, const W4Layout& l) const
    {
        const int64_t tiles = ((l.row_tiles + row_tiles - 1) / row_tiles) * ((a.M + rows - 1) / rows);
        const int64_t steps = turns ? (l.col_tiles + turns - 1) / turns : l.col_tiles;
        const int groups = kTileCols / a.group, words = groups * (a.scale_dtype == F32 ? 2 : 1);
        const float part = step_rows * (float)min(a.M, (int64_t)rows) / (float)rows + step_scales * (float)(words - 1) +
                           (a.has_zeros ? step_zeros * (float)groups : 0.0f);
        return start + (float)((tiles + 255) / 256) * (tile + (float)steps * (step + part));
    }
};

template <int G, typename TS, bool ZEROS>
hipError_t launch_gemm_form(const W4GemmArgs& a, const W4Layout& l, hipStream_t s)
{
    // (float32 scales of groups of 32 take too many registers beside three tiles; bfloat16 ones
    // with zero points keep nine in memory and still take 60 us where two tiles take 79, at 64 x
    // 41,024 x 4096, since all their workgroups run at once)
    constexpr int THREE = G == 32 && sizeof(TS) == 4 ? 2 : 3;
    constexpr int ANY = 1 << 30;
    constexpr W4Form kForms[] = {
        {16, 1, 0, 0, ANY, 2.86f, 0.081f, 0.063f, 0.051f, 0.0f, 0.004f},
        {16, 4, 2, 0, ANY, 2.91f, 0.386f, 0.307f, 0.0f, 0.024f, 0.033f},
        {32, 4, 2, 17, ANY, 2.61f, 0.865f, 0.440f, 0.0f, 0.026f, 0.051f},
        {16, 2, 4, 0, ANY, 2.89f, 0.428f, 0.328f, 0.0f, 0.026f, 0.029f},
        {32, 2, 4, 17, ANY, 1.35f, 2.16f, 0.552f, 0.0f, 0.028f, 0.046f},
        {32, THREE * 4, 2, 17, 32, 1.12f, 4.24f, 0.996f, 0.0f, -0.008f, 0.223f},
        {64, THREE * 4, 2, 33, ANY, 0.0f, 7.22f, 1.555f, 0.0f, -0.050f, 0.269f},
    };
    int best = 0;
    float least = kForms[0].cost(a, l);
    for (int f = 1; f < 7; ++f) {
        const float c = kForms[f].cost(a, l) * 1.05f;
        if (a.M >= kForms[f].least && a.M <= kForms[f].most && c < least) best = f, least = c;
    }
    switch (best) {
    case 0: return launch_gemm_tiles<2, G, TS, ZEROS>(a, l, s);
    case 1: return launch_gemm_rows<2, 1, 1, G, TS, ZEROS>(a, l, s);
    case 2: return launch_gemm_rows<2, 2, 1, G, TS, ZEROS>(a, l, s);
    case 3: return launch_gemm_rows<4, 1, 1, G, TS, ZEROS>(a, l, s);
    case 4: return launch_gemm_rows<4, 2, 1, G, TS, ZEROS>(a, l, s);
    case 5: return launch_gemm_rows<2, 2, THREE, G, TS, ZEROS>(a, l, s);
    default: return launch_gemm_rows<2, 4, THREE, G, TS, ZEROS>(a, l, s);
    }
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
