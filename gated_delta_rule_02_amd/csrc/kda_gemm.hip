// kda_gemm.hip -- C[M,N] = A[M,K] B[N,K]^T, bfloat16 inputs, float32 accumulate.
//
// The token mixer's dense projections ("Ling-3.1-flash: a 560B hybrid-attention
// MoE, counted from its safetensors headers", section "How KDA and MLA split the
// work": q, k, v, decay and gate 4096 -> 8192 and the output 8192 -> 4096, all
// full rank). Both operands are K-contiguous, which is exactly the layout the
// 16x16x32 bf16 MFMA consumes: each lane takes 8 consecutive K values of one
// row of A and one row of B.
//
// Two kernels of the plain product (the epilogue entry's forms stand below, with
// the rule that picks them). The main one (K a multiple of 64): a 256 x 256 tile of C per
// workgroup of 4 wavefronts, each owning 128 x 128 (8 x 8 MFMA tiles, 256
// accumulator registers: one wavefront per SIMD), K steps of 64 in two LDS
// stages filled by buffer-to-LDS copies of whole 128-byte operand rows (the
// copy of step k + 1 runs during step k). With K steps of 32 every copy
// request covered half a cache line, and the kernel issued twice the L2 read
// requests of the vendor BLAS for the same product; at the per-compute-unit
// limit on requests in flight that halved its operand bandwidth. The stage
// rows are 128 bytes with their 16-byte chunks XOR-swizzled by (row / 2) mod
// 8 (applied by choosing each lane's global source address: a buffer-to-LDS
// copy writes lane l to byte 16 l of its 1 KiB destination), so that the 16
// rows an MFMA operand read touches fall in distinct banks. The products are
// formed transposed (B tile x A tile^T): each lane then holds four
// consecutive columns of one row of C, stored with one 16-byte (float32) or
// 8-byte (bfloat16) access.
// The fallback (any K multiple of 8): 128 x 128 tiles, 2 x 2 wavefronts of
// 64 x 64, K steps of 32 through double-buffered LDS.
#include <cmath>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

// ------------------------------------------------------------ epilogue
// act(v + bias) + residual in float32. The activation and the residual's type
// are uniform over the launch: branches, not instantiations (a few scalar
// instructions per output against the K products before them).
__device__ __forceinline__ float activate(int act, float y)
{
    switch (act) {
        case 1: return y < 0.0f ? 0.0f : y;  // keeps NaN
        case 2: return siluf_(y);
        case 3: return 0.5f * y * (1.0f + erff(y * 0.70710678118654752f));
        case 4: return sigmoidf_(y);
        default: return y;
    }
}

// Workgroup -> tile of the epilogue entry's tiled kernels. Workgroup ids go round
// the 8 XCDs, each with an L2 of its own: every XCD takes one contiguous eighth of
// the tile list, and the list runs through the M tiles of a group of 8, then the
// N tiles, then the groups, so that the tiles of an XCD that run together share
// their rows of A and B.
__device__ __forceinline__ void xcd_tile(int tiles_m, int tiles_n, int& tm, int& tn)
{
    const int T = tiles_m * tiles_n, xcd = blockIdx.x & 7, per = T >> 3, rem = T & 7;
    const int tile = xcd * per + min(xcd, rem) + (int)(blockIdx.x >> 3);
    const int g = tile / (8 * tiles_n), rows = min(8, tiles_m - 8 * g), r = tile - g * 8 * tiles_n;
    tm = 8 * g + r % rows;
    tn = r / rows;
}

// Columns col .. col + 3 of a row's residual (0 past N).
__device__ __forceinline__ f32x4 residual4(const GemmArgs& a, int64_t row, int64_t col)
{
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    if (row >= a.M) return r;
    const int64_t i = row * a.ldr + col;
    const float* pf = static_cast<const float*>(a.res) + i;
    const bf16_t* pb = static_cast<const bf16_t*>(a.res) + i;
    if (col + 3 < a.N) return a.r_dtype == F32 ? ld4(pf) : ld4(pb);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < a.N) r[e] = a.r_dtype == F32 ? pf[e] : bf16_to_f32(pb[e]);
    return r;
}

// The epilogue of a wavefront's NI x NJ MFMA tiles (16 x 16, transposed: lane
// (m16, q4) element e of acc[i][j] is C[16i + m16][16j + 4q4 + e]), 16 rows at a
// time through LDS that the wavefront has to itself: a lane then holds four
// consecutive columns of a row that 4 NJ neighbouring lanes cover, so residual
// and C move in whole row segments, and the activation is a rolled loop (inlined
// into the unrolled tiles it spilled the 256 x 256 kernel's accumulators: 1,040
// registers, 15 times the time). The residual of the next 16 rows is
// loaded before this one's are finished.
template <int NJ> constexpr int kEpiFloats = 16 * (16 * NJ + 4);  // rows padded by 16 bytes
template <typename TC, int NI, int NJ>
__device__ __forceinline__ void tile_epilogue(const GemmArgs& a, const f32x4 (&acc)[NI][NJ], float* lds, int64_t row0,
                                              int64_t col0)
{
    constexpr int kLd = 16 * NJ + 4, kLanes = 4 * NJ, kRows = 64 / kLanes;  // kRows rows a step, NJ steps
    static_assert(64 % kLanes == 0, "whole rows a step");
    const int lane = threadIdx.x & 63, m16 = lane & 15, q4 = lane >> 4;
    const int r0 = lane / kLanes, c0 = 4 * (lane % kLanes);
    const int64_t col = col0 + c0;
    f32x4 bias = {0.f, 0.f, 0.f, 0.f};
    if (a.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < a.N) bias[e] = a.bias[col + e];
    }
    const bool whole = col + 3 < a.N;
    TC* Cp = static_cast<TC*>(a.C);
    f32x4 res[2][NJ];
    auto load_res = [&](int i, f32x4* r) {
#pragma unroll
        for (int t = 0; t < NJ; ++t) r[t] = residual4(a, row0 + 16 * i + r0 + kRows * t, col);
    };
    if (a.res) load_res(0, res[0]);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        wave_lds_order();  // the 16 rows before are read
#pragma unroll
        for (int j = 0; j < NJ; ++j) *reinterpret_cast<f32x4*>(lds + m16 * kLd + 16 * j + 4 * q4) = acc[i][j];
        wave_lds_order();
        if (a.res && i + 1 < NI) load_res(i + 1, res[(i + 1) & 1]);
        if (a.act) {
#pragma unroll 1
            for (int t = 0; t < NJ; ++t) {
                f32x4* p = reinterpret_cast<f32x4*>(lds + (r0 + kRows * t) * kLd + c0);
                f32x4 v = *p + bias;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = activate(a.act, v[e]);
                *p = v;
            }
        }
#pragma unroll
        for (int t = 0; t < NJ; ++t) {
            const int64_t row = row0 + 16 * i + r0 + kRows * t;
            f32x4 v = *reinterpret_cast<const f32x4*>(lds + (r0 + kRows * t) * kLd + c0);
            if (!a.act) v += bias;
            if (a.res) v += res[i & 1][t];
            if (row >= a.M) continue;
            TC* p = Cp + row * a.ldc + col;
            if (whole) {
                st4(p, v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < a.N) st(p + e, v[e]);
            }
        }
    }
}

constexpr int BM = 128, BN = 128, BK = 32;
constexpr int LDS_LD = BK + 8;  // padded row (bf16 elements)
constexpr int kThreads = 256;

__device__ __forceinline__ f32x4 mma32_bf16(const uint4& a, const uint4& b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <typename TC>
__global__ __launch_bounds__(kThreads) void gemm_kernel(GemmArgs a)
{
    __shared__ __attribute__((aligned(16))) bf16_t sA[2][BM][LDS_LD];
    __shared__ __attribute__((aligned(16))) bf16_t sB[2][BN][LDS_LD];

    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int m16 = lane & 15, q4 = lane >> 4;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const int64_t m0 = (int64_t)blockIdx.y * BM, n0 = (int64_t)blockIdx.x * BN;
    const bf16_t* A = static_cast<const bf16_t*>(a.A);
    const bf16_t* B = static_cast<const bf16_t*>(a.B);

    // global -> register staging: 2 x 16 B of A and of B per thread per K step
    uint4 ra[2], rb[2];
    auto gload = [&](int64_t k0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int idx = tid + j * kThreads;  // 0..511
            const int row = idx >> 2, kc = (idx & 3) * 8;
            const int64_t gm = m0 + row, gn = n0 + row, gk = k0 + kc;
            ra[j] = (gm < a.M && gk < a.K) ? *reinterpret_cast<const uint4*>(A + gm * a.lda + gk) : make_uint4(0, 0, 0, 0);
            rb[j] = (gn < a.N && gk < a.K) ? *reinterpret_cast<const uint4*>(B + gn * a.ldb + gk) : make_uint4(0, 0, 0, 0);
        }
    };
    auto sstore = [&](int buf) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int idx = tid + j * kThreads;
            const int row = idx >> 2, kc = (idx & 3) * 8;
            *reinterpret_cast<uint4*>(&sA[buf][row][kc]) = ra[j];
            *reinterpret_cast<uint4*>(&sB[buf][row][kc]) = rb[j];
        }
    };

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int nk = (int)((a.K + BK - 1) / BK);
    gload(0);
    sstore(0);
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
        const int buf = kt & 1;
        if (kt + 1 < nk) gload((int64_t)(kt + 1) * BK);
        uint4 fa[4], fb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) fa[i] = *reinterpret_cast<const uint4*>(&sA[buf][wm + 16 * i + m16][8 * q4]);
#pragma unroll
        for (int j = 0; j < 4; ++j) fb[j] = *reinterpret_cast<const uint4*>(&sB[buf][wn + 16 * j + m16][8 * q4]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mma32_bf16(fa[i], fb[j], acc[i][j]);
        if (kt + 1 < nk) sstore(buf ^ 1);
        __syncthreads();
    }

    TC* Cp = static_cast<TC*>(a.C);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t col = n0 + wn + 16 * j + m16;
            if (col >= a.N) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t row = m0 + wm + 16 * i + 4 * q4 + e;
                if (row < a.M) st(Cp + row * a.ldc + col, acc[i][j][e]);
            }
        }
}

// ------------------------------------------------------------ main kernel
constexpr int TM = 256, TN = 256, TK = 64;  // workgroup tile and K step (128 bytes of each operand row)
constexpr int kStageBytes = TM * TK * 2;     // one operand's stage: 256 rows x 128 B
typedef __attribute__((address_space(3))) void lds_void;

// LDS byte offset of 16-byte chunk c (0..7) of row r of a stage: the chunks are
// XOR-swizzled by (r / 2) mod 8. An operand read takes one chunk of 16
// consecutive rows; rows r and r + 1 lie in different halves of the 64
// banks and the 8 even (odd) rows get distinct slots, so the read touches
// every bank once.
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

// NJ: 16-column MFMA tiles per wavefront in N (8: the 256 x 256 tile; 2 or 4:
// a 256 x 64 or 256 x 128 tile for the last N mod 256 columns, so that they
// cost a fraction of a full tile instead of a whole one)
// EPI: the epilogue entry. TAIL (there, where K is any multiple of 8): K does not
// fill the last step; its chunks past K lie outside the descriptors, as zeros. A
// form of its own: the test in every step's copies costs 1.5 per cent of 8192 x
// 4096 x 8192.
template <typename TC, int NJ, bool EPI, bool TAIL>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm256_kernel(GemmArgs a)
{
    constexpr int TNW = 32 * NJ;         // columns of C per workgroup
    constexpr int kACopy = TM / 32;      // A copy instructions per wavefront and K step (8 rows each)
    constexpr int kBCopy = TNW / 32;     // B copy instructions per wavefront and K step
    static_assert(NJ == 2 || NJ == 4 || NJ == 8, "64, 128 or 256 columns");
    __shared__ __attribute__((aligned(16))) uint8_t smem[2][2][kStageBytes];  // [stage][A, B]
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m16 = lane & 15, q4 = lane >> 4;
    const int wm = (wave >> 1) * 128, wn = (wave & 1) * 16 * NJ;

    // tiles: consecutive workgroup ids run down a column of M tiles, so the
    // workgroups resident together share B tiles and a few A tiles
    const int tiles_m = (int)((a.M + TM - 1) / TM);
    int tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
    if constexpr (EPI) xcd_tile(tiles_m, (int)((a.N + TNW - 1) / TNW), tm, tn);
    const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TNW;

    // operand rows past M or N read as zero through the descriptor ranges
    const bf16_t* A = static_cast<const bf16_t*>(a.A) + m0 * a.lda;
    const bf16_t* B = static_cast<const bf16_t*>(a.B) + n0 * a.ldb;
    const int64_t rows_a = min<int64_t>(TM, a.M - m0), rows_b = min<int64_t>(TNW, a.N - n0);
    const rsrc_t ra = make_rsrc(A, ((rows_a - 1) * a.lda + a.K) * 2);
    const rsrc_t rb = make_rsrc(B, ((rows_b - 1) * a.ldb + a.K) * 2);

    // copy of K step kt into stage st: whole 128-byte rows, 8 rows per 1 KiB
    // instruction (lane l: row 8i + l/8, LDS chunk slot l%8, which holds the
    // row's K chunk slot ^ ((row / 2) mod 8))
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)&smem[0][0][0];
    const int lrow = lane >> 3, lslot = lane & 7;
    auto copy1 = [&](int kt, int st, int c) {  // copy c of the wavefront's kACopy + kBCopy
        const bool isa = c < kACopy;
        const int i = isa ? wave * kACopy + c : wave * kBCopy + c - kACopy;
        const int row = 8 * i + lrow;
        const int k = kt * TK + (lslot ^ ((row >> 1) & 7)) * 8;
        const int off = TAIL && k >= a.K ? (int)0x80000000 : (int)(row * (isa ? a.lda : a.ldb) * 2) + k * 2;
        lds_void* dst = (lds_void*)(uintptr_t)(lds0 + (st * 2 + (isa ? 0 : 1)) * kStageBytes + i * 1024);
        if (isa) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, dst, 16, off, 0, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, dst, 16, off, 0, 0, 0);
    };
    auto copy = [&](int kt, int st) {
#pragma unroll
        for (int c = 0; c < kACopy + kBCopy; ++c) copy1(kt, st, c);
    };
    const int nk = (int)((a.K + TK - 1) / TK);

    f32x4 acc[8][NJ];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Pipeline: two stages of 64 K. Step kt computes on stage kt % 2 (two K32
    // halves) while the copy of step kt + 1, issued at its start, fills the
    // other stage; the second half's fragments are read while the first half's
    // MFMAs run. At its end every wavefront waits for its copy (the compiler
    // does not track these copies: the wait is explicit) and the barrier
    // hands the stage over.
    if constexpr (EPI) {
        // The reads of one half run under the products of the other: the second half's
        // of step kt under the first's products, the first half's of step kt + 1 under
        // the second's. Between the two, once everyone has read all of stage kt and
        // its copy of step kt + 1 has landed, the stage is refilled with step kt + 2.
        u32x4_t fa[2][8], fb[2][NJ];
        auto read = [&](int st, int h, int c) {  // fragment c: the NJ of B, then the 8 of A
            if (c < NJ) fb[h][c] = *reinterpret_cast<const u32x4_t*>(&smem[st][1][0] + swz(wn + 16 * c + m16, 4 * h + q4));
            else fa[h][c - NJ] = *reinterpret_cast<const u32x4_t*>(&smem[st][0][0] + swz(wm + 16 * (c - NJ) + m16, 4 * h + q4));
        };
        constexpr int kRead = (8 + NJ + 7) / 8;           // reads beside each row of products (bunched 3 or 4: 1 to 2 per cent slower)
        constexpr int kCopy = (kACopy + kBCopy + 7) / 8;  // copies beside each row
        copy(0, 0);
        if (nk > 1) copy(1, 1);
        if (nk > 1) __builtin_amdgcn_s_waitcnt(0x0f70 | ((kACopy + kBCopy) & 15) | (((kACopy + kBCopy) >> 4) << 14));
        else __builtin_amdgcn_s_waitcnt(0x0f70);
        lds_barrier();
#pragma unroll
        for (int c = 0; c < NJ + 8; ++c) read(0, 0, c);
        for (int kt = 0; kt < nk; ++kt) {
            const int st = kt & 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[h][j]),
                                                                            __builtin_bit_cast(bf16x8, fa[h][i]),
                                                                            acc[i][j], 0, 0, 0);
                    // (the last step's read of a step that is not there is not used)
#pragma unroll
                    for (int c = kRead * i; c < min(kRead * (i + 1), NJ + 8); ++c) read(h ? st ^ 1 : st, h ^ 1, c);
                    if (h == 1 && kt + 2 < nk) {
#pragma unroll
                        for (int c = kCopy * i; c < min(kCopy * (i + 1), kACopy + kBCopy); ++c) copy1(kt + 2, st, c);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (h == 0) {
                    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
                    lds_barrier();
                }
            }
        }
        tile_epilogue<TC, 8, NJ>(a, acc, reinterpret_cast<float*>(&smem[0][0][0]) + wave * kEpiFloats<NJ>, m0 + wm,
                                 n0 + wn);
        return;
    }
    u32x4_t fa[8], fb[NJ];
    auto read_a = [&](int st, int h, int i) {
        fa[i] = *reinterpret_cast<const u32x4_t*>(&smem[st][0][0] + swz(wm + 16 * i + m16, 4 * h + q4));
    };
    auto read_b = [&](int st, int h, int j) {
        fb[j] = *reinterpret_cast<const u32x4_t*>(&smem[st][1][0] + swz(wn + 16 * j + m16, 4 * h + q4));
    };
    copy(0, 0);
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    lds_barrier();
    for (int kt = 0; kt < nk; ++kt) {
        const int st = kt & 1;
        if (kt + 1 < nk) copy(kt + 1, st ^ 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) read_a(st, 0, i);
#pragma unroll
        for (int j = 0; j < NJ; ++j) read_b(st, 0, j);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[j]),
                                                                        __builtin_bit_cast(bf16x8, fa[i]), acc[i][j], 0, 0, 0);
                if (h == 0) read_a(st, 1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (h == 0) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) read_b(st, 1, j);
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wavefront's copy has landed ...
        lds_barrier();                        // ... and everyone's; every read of stage st is done
    }

    // acc[i][j] holds C^T of tile (i, j): lane (m16, q4) element e is
    // C[row 16i + m16][column 16j + 4q4 + e]
    TC* Cp = static_cast<TC*>(a.C);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = m0 + wm + 16 * i + m16;
        if (row >= a.M) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int64_t col = n0 + wn + 16 * j + 4 * q4;
            TC* p = Cp + row * a.ldc + col;
            if (col + 3 < a.N) {
                if constexpr (sizeof(TC) == 4) {
                    *reinterpret_cast<f32x4*>(p) = acc[i][j];
                } else {
                    // float -> bfloat16 by the hardware conversion (round to nearest even)
                    const f32x4 v = acc[i][j];
                    typedef __bf16 b4_t __attribute__((ext_vector_type(4)));
                    *reinterpret_cast<b4_t*>(p) = b4_t{(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < a.N) st(p + e, acc[i][j][e]);
            }
        }
    }
}

// ------------------------------------------------------------ narrow kernel
// C[M, N <= 64] (the last N mod 256 columns of a wide product, such as the 64
// beta columns of the input projection): a 256 x 64 tile per workgroup leaves
// M / 256 workgroups, each walking all of K in latency-bound steps. Here a
// workgroup takes 32 rows and the four wavefronts split K four ways, each
// loading its operand fragments straight from memory into registers (a row's
// 128-byte line per 64-wide K step, the next step's fragments in flight during
// this step's products); the four partial tiles are summed through LDS.
constexpr int kNarrowRows = 32;

template <typename TC>
__global__ __launch_bounds__(256) void gemm_narrow_kernel(GemmArgs a)
{
    __shared__ f32x4 part[3][2][4][64];  // the partial tiles of wavefronts 1 .. 3
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m16 = lane & 15, q4 = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * kNarrowRows;
    const int64_t rows_a = min<int64_t>(kNarrowRows, a.M - m0);
    const rsrc_t ra = make_rsrc(static_cast<const bf16_t*>(a.A) + m0 * a.lda, ((rows_a - 1) * a.lda + a.K) * 2);
    const rsrc_t rb = make_rsrc(a.B, ((a.N - 1) * a.ldb + a.K) * 2);
    const int kq = (int)(a.K / 4);                  // this wavefront's K range: [wave kq, (wave + 1) kq)
    const int nk = kq / 64;
    // lane (m16, q4): row 16 i + m16, K elements 8 q4 .. +7 of each 32-wide half
    int offa[2], offb[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) offa[i] = (int)((16 * i + m16) * a.lda * 2) + (wave * kq + 8 * q4) * 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) offb[j] = (int)((16 * j + m16) * a.ldb * 2) + (wave * kq + 8 * q4) * 2;
    u32x4_t fa[2][2][2], fb[2][4][2];  // [buffer][tile][K half]
    auto load = [&](int kt, int buf) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                fa[buf][i][h] = __builtin_amdgcn_raw_buffer_load_b128(ra, offa[i], (kt * 64 + 32 * h) * 2, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fb[buf][j][h] = __builtin_amdgcn_raw_buffer_load_b128(rb, offb[j], (kt * 64 + 32 * h) * 2, 0);
        }
    };
    f32x4 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    load(0, 0);
    for (int kt = 0; kt < nk; kt += 2) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (kt + b >= nk) break;
            if (kt + b + 1 < nk) load(kt + b + 1, b ^ 1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, fb[b][j][h]), __builtin_bit_cast(bf16x8, fa[b][i][h]), acc[i][j],
                            0, 0, 0);
        }
    }
    // acc[i][j] holds C^T of tile (i, j): lane (m16, q4) element e is
    // C[row 16i + m16][column 16j + 4q4 + e]; wavefronts 1 .. 3 hand theirs to 0
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[wave - 1][i][j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += part[w][i][j][lane];
    TC* Cp = static_cast<TC*>(a.C);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = m0 + 16 * i + m16;
        if (row >= a.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t col = 16 * j + 4 * q4;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.N) st(Cp + row * a.ldc + col + e, acc[i][j][e]);
        }
    }
}

// ------------------------------------------------------------ general tiles
// The epilogue entry's kernel for every shape the 256 x 256 tiles do not suit:
// TMx x TNx tiles of C by WM x WN wavefronts, K steps of 64 in STAGES LDS stages
// filled by buffer-to-LDS copies STAGES - 1 steps ahead (the last of them may
// still be in flight while a step computes: the wait counts copies). Rows past
// M or N and, in the last step, chunks past K lie outside the descriptors and
// read as zero.
template <typename TC, int TMx, int TNx, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM * WN * 64) void gemm_tile_kernel(GemmArgs a)
{
    constexpr int kW = WM * WN, NI = TMx / WM / 16, NJ = TNx / WN / 16;
    constexpr int kStage = (TMx + TNx) * 128;             // bytes of a stage: A rows, then B rows, 128 bytes each
    constexpr int kCopies = (TMx + TNx) / 8 / kW;         // 1 KiB copies per wavefront and stage
    static_assert((TMx + TNx) % (8 * kW) == 0 && TMx % 8 == 0, "whole copies");
    static_assert(kW * kEpiFloats<NJ> * 4 <= STAGES * kStage, "the epilogue fits the stages");
    __shared__ __attribute__((aligned(16))) uint8_t smem[STAGES * kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m16 = lane & 15, q4 = lane >> 4;
    const int wm = (wave / WN) * (TMx / WM), wn = (wave % WN) * (TNx / WN);
    const int tiles_m = (int)((a.M + TMx - 1) / TMx);
    int tm, tn;
    xcd_tile(tiles_m, (int)((a.N + TNx - 1) / TNx), tm, tn);
    const int64_t m0 = (int64_t)tm * TMx, n0 = (int64_t)tn * TNx;
    const int64_t rows_a = min<int64_t>(TMx, a.M - m0), rows_b = min<int64_t>(TNx, a.N - n0);
    const rsrc_t ra = make_rsrc(static_cast<const bf16_t*>(a.A) + m0 * a.lda, ((rows_a - 1) * a.lda + a.K) * 2);
    const rsrc_t rb = make_rsrc(static_cast<const bf16_t*>(a.B) + n0 * a.ldb, ((rows_b - 1) * a.ldb + a.K) * 2);

    // copy i (of this wavefront's kCopies): rows 8i .. 8i + 7 of the stage, lane
    // l its row l / 8, LDS chunk l % 8 (K chunk swizzled as the main kernel's)
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)&smem[0];
    const int lrow = lane >> 3, lslot = lane & 7;
    const int nk = (int)((a.K + 63) / 64);
    auto copy = [&](int kt) {
        const int st = kt % STAGES;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
            const int row = 8 * (wave * kCopies + c);  // of A rows then B rows; a copy lies in one of them
            const bool isa = row < TMx;
            const int r = (isa ? row : row - TMx) + lrow;
            const int k = kt * 64 + (lslot ^ ((r >> 1) & 7)) * 8;
            const int64_t ld = isa ? a.lda : a.ldb;
            const int64_t rows = isa ? rows_a : rows_b;
            const int off = k < a.K && r < rows ? (int)((r * ld + k) * 2) : (int)0x80000000;  // outside either descriptor
            lds_void* dst = (lds_void*)(uintptr_t)(lds0 + st * kStage + row * 128);
            if (isa) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, dst, 16, off, 0, 0, 0);
            else __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, dst, 16, off, 0, 0, 0);
        }
    };
    f32x4 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < STAGES - 1; ++p)
        if (p < nk) copy(p);
    for (int kt = 0; kt < nk; ++kt) {
        // stage kt is there once at most the copies of the later steps under way are left
        constexpr int kAhead = (STAGES - 2) * kCopies;
        if (kt + STAGES - 1 <= nk) __builtin_amdgcn_s_waitcnt(0x0f70 | (kAhead & 15) | ((kAhead >> 4) << 14));
        else __builtin_amdgcn_s_waitcnt(0x0f70);  // the last steps: everything
        lds_barrier();  // everyone's copies of stage kt; every read of the stage refilled now is done
        if (kt + STAGES - 1 < nk) copy(kt + STAGES - 1);
        const uint8_t* sa = smem + (kt % STAGES) * kStage;
        const uint8_t* sb = sa + TMx * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4_t fa[NI], fb[NJ];
#pragma unroll
            for (int i = 0; i < NI; ++i) fa[i] = *reinterpret_cast<const u32x4_t*>(sa + swz(wm + 16 * i + m16, 4 * h + q4));
#pragma unroll
            for (int j = 0; j < NJ; ++j) fb[j] = *reinterpret_cast<const u32x4_t*>(sb + swz(wn + 16 * j + m16, 4 * h + q4));
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[j]),
                                                                        __builtin_bit_cast(bf16x8, fa[i]), acc[i][j], 0,
                                                                        0, 0);
        }
    }
    lds_barrier();  // every wavefront has read its last stage
    tile_epilogue<TC, NI, NJ>(a, acc, reinterpret_cast<float*>(smem) + wave * kEpiFloats<NJ>, m0 + wm, n0 + wn);
}

// ------------------------------------------------------------ small tiles, K split
// 16 MT x 16 NT tiles of C by KS wavefronts that split K: wavefront w takes the
// K steps w, w + KS, ... of 64 on its own, through its own ring of S LDS stages, so
// that the loop has no barrier, a fragment read from LDS serves MT (NT) products,
// and every wavefront keeps S - 1 steps of loads under way. What bounds it is how
// fast a compute unit takes in the (16 MT + 16 NT) rows of its tile, so the
// launcher picks the tile that gives every compute unit the fewest bytes. The
// partial tiles are summed in LDS in a fixed order, a row of MFMA tiles per
// wavefront. Rows past M or N and chunks past K lie outside the descriptors and
// read as zero.
template <typename TC, int MT, int NT, int KS, int S>
__global__ __launch_bounds__(KS * 64) void gemm_ring_kernel(GemmArgs a)
{
    constexpr int kStage = (MT + NT) * 2048;      // bytes: 16 (MT + NT) rows of 128
    constexpr int kRing = S * kStage, kPart = MT * NT * 1024;
    constexpr int kCopies = 2 * (MT + NT);        // 1 KiB copies per stage
    static_assert(kPart + kEpiFloats<NT> * 4 <= kRing, "a partial tile and the epilogue's rows fit the ring");
    static_assert(KS * kRing <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(16))) uint8_t smem[KS * kRing];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m16 = lane & 15, q4 = lane >> 4;
    int tm, tn;
    xcd_tile((int)((a.M + 16 * MT - 1) / (16 * MT)), (int)((a.N + 16 * NT - 1) / (16 * NT)), tm, tn);
    const int64_t m0 = (int64_t)tm * 16 * MT, n0 = (int64_t)tn * 16 * NT;
    const int rows_a = (int)min<int64_t>(16 * MT, a.M - m0), rows_b = (int)min<int64_t>(16 * NT, a.N - n0);
    const rsrc_t ra = make_rsrc(static_cast<const bf16_t*>(a.A) + m0 * a.lda, ((rows_a - 1) * a.lda + a.K) * 2);
    const rsrc_t rb = make_rsrc(static_cast<const bf16_t*>(a.B) + n0 * a.ldb, ((rows_b - 1) * a.ldb + a.K) * 2);
    uint8_t* ring = smem + wave * kRing;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)ring;
    const int lrow = lane >> 3, lslot = lane & 7;
    const int nk = (int)((a.K + 63) / 64), mine = (nk - wave + KS - 1) / KS;  // this wavefront's steps
    auto copy = [&](int i) {
        const int kt = wave + i * KS, st = i % S;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
            const bool isa = c < 2 * MT;
            const int r = 8 * (isa ? c : c - 2 * MT) + lrow;
            const int k = kt * 64 + (lslot ^ ((r >> 1) & 7)) * 8;
            const int off = k < a.K && r < (isa ? rows_a : rows_b) ? (int)((r * (isa ? a.lda : a.ldb) + k) * 2)
                                                                   : (int)0x80000000;  // outside either descriptor
            lds_void* dst = (lds_void*)(uintptr_t)(lds0 + st * kStage + c * 1024);
            if (isa) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, dst, 16, off, 0, 0, 0);
            else __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, dst, 16, off, 0, 0, 0);
        }
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < S - 1; ++p)
        if (p < mine) copy(p);
    for (int i = 0; i < mine; ++i) {
        // this step's copies have landed (the later steps' may be under way), and
        // the last step's fragments, whose stage is refilled now, are read
        constexpr int kAhead = (S - 2) * kCopies;
        static_assert(kAhead < 64, "copies the wait can count");
        asm volatile("" ::: "memory");
        if (i + S - 1 <= mine) __builtin_amdgcn_s_waitcnt(0x0070 | (kAhead & 15) | ((kAhead >> 4) << 14));
        else __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        asm volatile("" ::: "memory");
        if (i + S - 1 < mine) copy(i + S - 1);
        const uint8_t* sa = ring + (i % S) * kStage;
        const uint8_t* sb = sa + MT * 2048;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4_t fa[MT], fb[NT];
#pragma unroll
            for (int m = 0; m < MT; ++m) fa[m] = *reinterpret_cast<const u32x4_t*>(sa + swz(16 * m + m16, 4 * h + q4));
#pragma unroll
            for (int n = 0; n < NT; ++n) fb[n] = *reinterpret_cast<const u32x4_t*>(sb + swz(16 * n + m16, 4 * h + q4));
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[n]),
                                                                        __builtin_bit_cast(bf16x8, fa[m]), acc[m][n], 0,
                                                                        0, 0);
        }
    }
    // every wavefront's partial tile at the start of its ring
    f32x4* part = reinterpret_cast<f32x4*>(ring);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) part[(m * NT + n) * 64 + lane] = acc[m][n];
    lds_barrier();
#pragma unroll 1
    for (int m = wave; m < MT; m += KS) {
        f32x4 sum[1][NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            sum[0][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < KS; ++w)
                sum[0][n] += *reinterpret_cast<const f32x4*>(smem + w * kRing + ((m * NT + n) * 64 + lane) * 16);
        }
        tile_epilogue<TC, 1, NT>(a, sum, reinterpret_cast<float*>(ring + kPart), m0 + 16 * m, n0);
    }
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& a, hipStream_t s)
{
    // the main kernel's copies address rows through 32-bit offsets
    const bool main_path = a.K % 64 == 0 && (int64_t)TM * a.lda * 2 < ((int64_t)1 << 31) &&
                           (int64_t)TN * a.ldb * 2 < ((int64_t)1 << 31);
    if (main_path) {
        // whole 256-column tiles, then the last N mod 256 columns in 64- or
        // 128-column tiles (the 64 columns of the beta projection in the
        // 41,024-wide input projection: one more round of 32 workgroups)
        const int64_t tiles_m = (a.M + TM - 1) / TM;
        GemmArgs m = a;
        m.N = a.N / TN * TN;
        if (m.N > 0) {
            dim3 grid((unsigned)(tiles_m * (m.N / TN))), block(256);
            if (a.c_dtype == F32) hipLaunchKernelGGL((gemm256_kernel<float, 8, false, false>), grid, block, 0, s, m);
            else hipLaunchKernelGGL((gemm256_kernel<bf16_t, 8, false, false>), grid, block, 0, s, m);
        }
        GemmArgs r = a;
        r.N = a.N - m.N;
        if (r.N > 0 && r.N <= 64 && a.K % 256 == 0) {
            // up to 64 columns left: 32-row workgroups with K split four ways
            r.B = static_cast<const bf16_t*>(a.B) + m.N * a.ldb;
            r.C = static_cast<uint8_t*>(a.C) + m.N * (a.c_dtype == F32 ? 4 : 2);
            const dim3 grid((unsigned)((a.M + kNarrowRows - 1) / kNarrowRows)), block(256);
            if (a.c_dtype == F32) hipLaunchKernelGGL((gemm_narrow_kernel<float>), grid, block, 0, s, r);
            else hipLaunchKernelGGL((gemm_narrow_kernel<bf16_t>), grid, block, 0, s, r);
        } else if (r.N > 0) {
            r.B = static_cast<const bf16_t*>(a.B) + m.N * a.ldb;
            r.C = static_cast<uint8_t*>(a.C) + m.N * (a.c_dtype == F32 ? 4 : 2);
            const int nj = r.N <= 64 ? 2 : (r.N <= 128 ? 4 : 8);
            dim3 grid((unsigned)(tiles_m * ((r.N + 32 * nj - 1) / (32 * nj)))), block(256);
#define KDA_GEMM_REM(NJ)                                                                            \
    if (a.c_dtype == F32) hipLaunchKernelGGL((gemm256_kernel<float, NJ, false, false>), grid, block, 0, s, r);     \
    else hipLaunchKernelGGL((gemm256_kernel<bf16_t, NJ, false, false>), grid, block, 0, s, r);
            if (nj == 2) { KDA_GEMM_REM(2) }
            else if (nj == 4) { KDA_GEMM_REM(4) }
            else { KDA_GEMM_REM(8) }
#undef KDA_GEMM_REM
        }
        return hipGetLastError();
    }
    dim3 grid((unsigned)((a.N + BN - 1) / BN), (unsigned)((a.M + BM - 1) / BM)), block(kThreads);
    if (a.c_dtype == F32)
        hipLaunchKernelGGL(gemm_kernel<float>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(gemm_kernel<bf16_t>, grid, block, 0, s, a);
    return hipGetLastError();
}

namespace {

template <typename TC, int TMx, int TNx, int WM, int WN, int STAGES>
hipError_t launch_tile(const GemmArgs& a, hipStream_t s)
{
    const int64_t tiles = ((a.M + TMx - 1) / TMx) * ((a.N + TNx - 1) / TNx);
    hipLaunchKernelGGL((gemm_tile_kernel<TC, TMx, TNx, WM, WN, STAGES>), dim3((unsigned)tiles), dim3(WM * WN * 64), 0, s, a);
    return hipGetLastError();
}

template <typename TC>
hipError_t launch_256(const GemmArgs& a, hipStream_t s)
{
    const int64_t tiles = ((a.M + TM - 1) / TM) * ((a.N + TN - 1) / TN);
    if (a.K % TK) hipLaunchKernelGGL((gemm256_kernel<TC, 8, true, true>), dim3((unsigned)tiles), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((gemm256_kernel<TC, 8, true, false>), dim3((unsigned)tiles), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename TC, int MT, int NT, int KS, int S>
hipError_t launch_ring(const GemmArgs& a, hipStream_t s)
{
    const int64_t tiles = ((a.M + 16 * MT - 1) / (16 * MT)) * ((a.N + 16 * NT - 1) / (16 * NT));
    hipLaunchKernelGGL((gemm_ring_kernel<TC, MT, NT, KS, S>), dim3((unsigned)tiles), dim3(KS * 64), 0, s, a);
    return hipGetLastError();
}

// The form with the least cost: rounds of tiles over the 256 compute units, times what a
// tile costs: the rows of A and B that it takes in, K values each, at a rate relative to
// the K-split tiles', plus what starts and ends it (the first loads' latency, the
// epilogue) in the same unit (60,000 is about 2 us). Both numbers are fitted to the
// times of every form at 365 sizes (1 to 8,192 rows, 36 to 41,024 columns, K 136 to
// 8,192), where this choice is 0.9 per cent (geometric mean) above the best form, and
// 1.8 at 365 others. The
// tiles that are bound by taking their rows in cost about their rows; the 256 x 256
// ones are bound by the matrix instructions instead, are the only ones past 1.1
// PFLOP/s (1.3 at 8192 rows), and pay most at their ends (one wavefront a SIMD). Left out of the list, a
// form costs over all sizes: 16 x 16 4 per cent, 32 x 32, 64 x 64, 128 x 128 and
// 192 x 128 1 each, the others 0.2 to 0.7; 32 x 16, 32 x 64, 128 x 64 and 128 x 256 tiles
// gave less than 0.1 and are not built. 4096 columns, K = 8192, us, this choice | the
// next best of the list: 1 row 13.8 | 14.9, 64 rows 19.9 | 26.4, 96 rows 22.6 | 30.9, 192 rows
// 31.9 | 34.6, 333 rows 39.3 | 58.2, 1024 rows 77.0 | 94.6, 2048 rows 129 | 150, 3000
// rows 182 | 204, 4096 rows 208 | 261.
template <typename TC>
hipError_t launch_epilogue(const GemmArgs& a, hipStream_t s)
{
    struct Form {
        int tm, tn;
        float row, ends;
        hipError_t (*launch)(const GemmArgs&, hipStream_t);
    };
    static const Form forms[] = {
        {16, 16, 1.0f, 60e3f, launch_ring<TC, 1, 1, 8, 4>},
        {16, 32, 1.0f, 60e3f, launch_ring<TC, 1, 2, 4, 6>},
        {32, 32, 1.0f, 60e3f, launch_ring<TC, 2, 2, 4, 4>},
        {64, 32, 1.0f, 60e3f, launch_ring<TC, 4, 2, 4, 3>},
        {48, 64, 1.0f, 60e3f, launch_ring<TC, 3, 4, 4, 2>},
        {64, 64, 1.0f, 60e3f, launch_ring<TC, 4, 4, 4, 2>},
        {96, 64, 1.05f, 120e3f, launch_ring<TC, 6, 4, 4, 2>},
        {128, 128, 1.1f, 100e3f, launch_tile<TC, 128, 128, 4, 2, 4>},
        {192, 128, 1.15f, 140e3f, launch_tile<TC, 192, 128, 4, 2, 3>},
        {256, 128, 1.15f, 240e3f, launch_tile<TC, 256, 128, 4, 2, 3>},
        {256, 256, 1.3f, 600e3f, launch_256<TC>},
    };
    const Form* best = nullptr;
    double least = 0.0;
    for (const Form& f : forms) {
        const double tiles = (double)((a.M + f.tm - 1) / f.tm) * (double)((a.N + f.tn - 1) / f.tn);
        const double cost = std::ceil(tiles / 256.0) * ((f.tm + f.tn) * f.row * (double)a.K + f.ends);
        if (!best || cost < least) best = &f, least = cost;
    }
    return best->launch(a, s);
}

}  // namespace

hipError_t launch_gemm_epilogue(const GemmArgs& a, hipStream_t s)
{
    return a.c_dtype == F32 ? launch_epilogue<float>(a, s) : launch_epilogue<bf16_t>(a, s);
}

}  // namespace kda
