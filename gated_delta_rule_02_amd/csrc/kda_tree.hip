// kda_tree.hip -- verification of trees of drafted tokens (gfx950): the
// recurrence and the prologue convolution along every root path of a tree, and
// the commit of the accepted path.
//
// A tree of N <= 64 nodes hangs below a sequence's state: parents[i] is -1 (the
// state itself) or a node before i. Any other value marks node i as absent, and
// with it every node below it: no result depends on it, its outputs are zero,
// and committing it changes nothing.
//
// With S0 the state, D(i, j) the product of the retentions alpha over the path
// from j (excluded) down to i, and D(i) the same from the state, the recurrence
// S_i = (I - beta_i k_i k_i^T) Diag(alpha_i) S_p(i) + beta_i k_i v_i^T unrolls to
//   u_i = beta_i (v_i - S0^T (D(i) k_i) - sum_j [k_i . D(i, j) k_j] u_j)    j above i
//   o_i = scale (S0^T (D(i) q_i) + sum_j [q_i . D(i, j) k_j] u_j)           j above i, and i
//   S_i = Diag(D(i)) S0 + sum_j (D(i, j) k_j) u_j^T                          j above i, and i
// so all nodes read S0 once, no state but S0 is formed, and the writes u of the
// accepted path are all that a commit needs. The decays are products of the
// alphas taken along the path, never quotients: exact for every floor down to
// -inf, and a path that has decayed to nothing contributes nothing.
#include <utility>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int D = 128;

// The parent of this lane's node: -1 (the state), a node, or -2 (absent, itself
// or through a node above it). Every lane of the wavefront takes part.
__device__ __forceinline__ int load_parent(const int32_t* parents, int N)
{
    const int lane = threadIdx.x & 63;
    return lane < N ? parents[lane] : -2;
}
__device__ __forceinline__ int tree_parent(int p)  // p: load_parent()
{
    if (p < -1 || p >= (int)(threadIdx.x & 63)) p = -2;
    // pointer doubling: after s steps `up` is the 2^s-th node above, or -1 / -2
    int up = p;
#pragma unroll
    for (int s = 0; s < 6; ++s) {
        const int far = __shfl(up, max(up, 0), 64);
        if (up >= 0) up = far;
    }
    return up == -2 ? -2 : p;
}

// Sum over aligned groups of 16 lanes, in every lane (rotations within the row).
template <int ROR>
__device__ __forceinline__ float add_ror(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + ROR, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum16(float v) { return add_ror<1>(add_ror<2>(add_ror<4>(add_ror<8>(v)))); }

// ------------------------------------------------------------ convolution
template <typename T>
__device__ __forceinline__ void row8(const T* p, float* f)
{
    if constexpr (sizeof(T) == 2) {
        Vec16<bf16_t>::unpack(ld16(p), f);
    } else {
        Vec16<float>::unpack(ld16(p), f);
        Vec16<float>::unpack(ld16(p + 4), f + 4);
    }
}
template <typename T>
__device__ __forceinline__ void put8(T* p, const float* f)
{
    if constexpr (sizeof(T) == 2) {
        st16(p, Vec16<bf16_t>::pack(f));
    } else {
        st16(p, Vec16<float>::pack(f));
        st16(p + 4, Vec16<float>::pack(f + 4));
    }
}

// Rows of a sequence as one list: its W - 1 history rows, then its nodes. From a
// node (>= 0) or history row (< 0, -1 the newest) `at`, the input one step back
// is the node above it or the next older history row; `at + W - 1` indexes the list.
__device__ __forceinline__ int step_back(int parent, int at)
{
    const int up = __shfl(parent, max(at, 0), 64);
    return at >= 0 ? up : at - 1;
}
template <typename T>
__device__ __forceinline__ const T* list_row(const T* x, int64_t x_ld, const T* hist, int C, int W, int at)
{
    return at >= 0 ? x + at * x_ld : hist + (size_t)(W - 1 + at) * C;
}

// A workgroup takes 512 channels (8 a lane) of one sequence: all of its rows, history
// and nodes, go to LDS in one sweep that does not wait for the tree (R rows at
// most), each row read from memory once; meanwhile every wavefront resolves the
// tree; then the wavefronts take the nodes in turn, each node's W rows from LDS.
// (Reading each node's window from memory instead, four nodes a workgroup, was
// bound by the repeated reads: 16.8 against 11.2 us for 64 trees of 16 nodes, 8,192
// channels.)
template <typename T, int W, int R>
__global__ __launch_bounds__(256) void conv_tree_kernel(ConvTreeArgs a)
{
    using V = Vec16<T>;
    constexpr int NV = 8 / V::N;  // 16-byte vectors per 8 channels
    constexpr int kBatch = 8 / NV;
    __shared__ u32x4_t s_x[R][NV][64];
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int parent_in = load_parent(a.parents + (size_t)b * a.N, a.N);
    // The lanes hold the tree: none of them may leave before the last readlane
    // (a lane that has left has no value to read). Lanes past C work on the
    // slab's first channels and store nothing.
    const int slab = blockIdx.y * 512;
    const bool in = slab + 8 * lane < a.C;  // C is a multiple of 128: whole 16-lane groups
    const int c = in ? slab + 8 * lane : slab;
    const T* x = static_cast<const T*>(a.x) + (size_t)b * a.N * a.x_ld + c;
    const T* hist = static_cast<const T*>(a.hist) + (size_t)b * (W - 1) * a.C + c;
    const int rows = W - 1 + a.N;  // row r of the list: history r, then node r - (W - 1)
    for (int r0 = wave; r0 < rows; r0 += 4 * kBatch) {
        u32x4_t v[kBatch][NV];
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const T* p = list_row(x, a.x_ld, hist, a.C, W, min(r0 + 4 * n, rows - 1) - (W - 1));
#pragma unroll
            for (int q = 0; q < NV; ++q) v[n][q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + q * V::N));
        }
#pragma unroll
        for (int n = 0; n < kBatch; ++n)
            if (r0 + 4 * n < rows)
#pragma unroll
                for (int q = 0; q < NV; ++q) s_x[r0 + 4 * n][q][lane] = v[n][q];
    }
    float w[8 * W], bias[8];
#pragma unroll
    for (int v = 0; v < W; ++v) row8(static_cast<const T*>(a.weight) + (size_t)c * W + 8 * v, w + 8 * v);
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = 0.0f;
    if (a.bias) row8(static_cast<const T*>(a.bias) + c, bias);
    // taps of every node, each lane its own node: tap j reads list row tap[j] + W - 1
    const int parent = tree_parent(parent_in);
    int tap[W];
    tap[W - 1] = lane;
#pragma unroll
    for (int j = W - 2; j >= 0; --j) tap[j] = step_back(parent, tap[j + 1]);
    lds_barrier();
    for (int i = wave; i < a.N; i += 4) {
        float acc[8];
        if (__builtin_amdgcn_readlane(parent, i) == -2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = bias[e];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int r = __builtin_amdgcn_readlane(tap[j], i) + W - 1;
                float f[8];
#pragma unroll
                for (int q = 0; q < NV; ++q) V::unpack(s_x[r][q][lane], f + q * V::N);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += w[e * W + j] * f[e];
            }
            if (a.apply_silu) {
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = siluf_(acc[e]);
            }
            if (a.l2_group) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += acc[e] * acc[e];
                const float r = rsqrtf(sum16(ss) + a.l2_eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] *= r;
            }
        }
        if (in) put8(static_cast<T*>(a.y) + ((size_t)b * a.N + i) * a.C + c, acc);
    }
}

// hist <- the last W - 1 inputs up to the accepted node (bit copies). A thread
// reads all of its channels' rows before it writes one: in place.
template <typename T, int W>
__global__ __launch_bounds__(256) void conv_commit_kernel(ConvTreeArgs a)
{
    constexpr int NV = 8 * (int)sizeof(T) / 16;
    const int b = blockIdx.x;
    const int parent = tree_parent(load_parent(a.parents + (size_t)b * a.N, a.N));
    const int acc = a.accepted[b];
    if (acc < 0 || acc >= a.N || __builtin_amdgcn_readlane(parent, acc & 63) == -2) return;  // uniform
    int at[W - 1];
    at[W - 2] = acc;
#pragma unroll
    for (int j = W - 3; j >= 0; --j) at[j] = step_back(parent, at[j + 1]);
    const int c = blockIdx.y * 2048 + 8 * threadIdx.x;
    if (c >= a.C) return;  // from here every lane has the rows it needs in its own registers
    const T* x = static_cast<const T*>(a.x) + (size_t)b * a.N * a.x_ld + c;
    T* hist = static_cast<T*>(a.hist) + (size_t)b * (W - 1) * a.C + c;
    u32x4_t row[W - 1][NV];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const T* p = list_row<T>(x, a.x_ld, hist, a.C, W, at[j]);
#pragma unroll
        for (int v = 0; v < NV; ++v) row[j][v] = ld16(p + v * Vec16<T>::N);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int v = 0; v < NV; ++v) st16(hist + (size_t)j * a.C + v * Vec16<T>::N, row[j][v]);
}

// ------------------------------------------------------------ verification
// One workgroup per (sequence, head), of NW wavefronts that take 128 / NW value
// channels each. Four phases:
//   load   the nodes' inputs, then the wavefront's columns of S0 into registers:
//          used last, so that the work up to the products runs while they arrive;
//   walk   16 lanes per node walk up its path with the running decay, forming
//          the node's products with every node above it (P with q_i, A with k_i)
//          and, at the end, the decayed rows D(i) k_i and D(i) q_i. Only pairs on
//          a path are formed;
//   read   [D k; D q] S0 on the float32 matrix instruction (float32 products
//          and sums: the results are held to float32 accuracy), rows from LDS, S0
//          from the registers;
//   solve  u by forward substitution in blocks of 16 nodes: the blocks before
//          by the matrix instruction on the accumulators that hold (D k) S0 - v,
//          then within the block each lane a value channel, the block's
//          remainders in registers (after u_j every r_i takes - A_ij u_j,
//          independent operations); then o += P u by the matrix instruction on
//          the accumulators that hold (D q) S0.
// What bounds it (float32 states, 64 heads): up to 16 nodes HBM, 128 trees of 16
// nodes 151 us = 5.3 TB/s (a copy reaches 5.1), 64 of 8 nodes 54 us = 6.1 TB/s;
// above, the walk (with it skipped, 64 trees of 32 nodes took 115 of 188 us, 32 of 64
// nodes 166 of 320, before the forms below) and the products. Now 64 of 32 nodes 148 us, 64 of
// 40 258 us, 32 of 64 263 us. bfloat16 states take about the same: 128 of 16 nodes 145 us,
// 64 of 32 145 us, 64 of 40 258 us, 32 of 64 261 us. Tried and slower up to 32 nodes:
// all pairs at once as a matrix product of rows scaled by exp(G + C) and exp(-G - C),
// C a center per channel (128 of 16 nodes 157 | 180 us; the loads before the state's
// get more and smaller).
// NP: N rounded up to 8, 16, 32, 48 or 64.
// NW wavefronts: 4, and 8 for NP > 32, where a compute unit holds one or two
// workgroups and 4 wavefronts each left a SIMD with too few to cover the latencies of the
// walk and the substitution (32 trees of 64 nodes 320 | 275 us with 4 | 8; 64 of 32 nodes
// 178 | 189, so 4 there).
template <int NP> constexpr int kTreeWaves = tree_threads(NP) / 64;
template <int NP> constexpr int kTreePerSimd = NP <= 16 || NP == 48 ? 4 : (NP == 32 ? 3 : 2);  // wavefronts per SIMD (by LDS and registers)

// f(0), ..., f(N - 1) with compile-time arguments: indexes of register arrays are
// constants from the start (a loop unrolled late left the remainders of the
// substitution in one tuple of registers, copied and spilled at every update).
template <typename F, int... I>
__device__ __forceinline__ void static_for(F&& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f)
{
    static_for(f, std::make_integer_sequence<int, N>{});
}

// Four, or CT (1 or 2), consecutive values as they are stored, and as floats.
template <int CT> using cols_t = float __attribute__((ext_vector_type(CT)));
template <typename T, int CT> struct Raw;
template <int CT> struct Raw<float, CT> {
    typedef f32x4 R4;
    typedef cols_t<CT> RC;
    __device__ static f32x4 f4(const R4& v) { return v; }
    __device__ static cols_t<CT> fc(const RC& v) { return v; }
};
template <int CT> struct Raw<bf16_t, CT> {
    typedef uint2 R4;
    typedef uint16_t RC __attribute__((ext_vector_type(CT)));
    __device__ static f32x4 f4(const uint2& u)
    {
        return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u)};
    }
    __device__ static cols_t<CT> fc(const RC& u)
    {
        cols_t<CT> f;
#pragma unroll
        for (int c = 0; c < CT; ++c) f[c] = bf16_to_f32(u[c]);
        return f;
    }
};

template <typename TIN, typename TOUT, typename TS, int NP>
__global__ __launch_bounds__(64 * kTreeWaves<NP>, kTreePerSimd<NP>) void decode_tree_kernel(TreeArgs a)
{
    constexpr int NW = kTreeWaves<NP>, CT = 8 / NW, CW = 16 * CT;  // value channels: CT column tiles a wavefront
    constexpr bool kAhead = NP == 64 || (NP <= 32 && sizeof(TS) == 2);  // (elsewhere the registers do not suffice)
    typedef cols_t<CT> cols;
    constexpr int LP = NP + 4;
    constexpr int MT = 2 * NP / 16;            // row tiles: D k, then D q (NP = 8: one tile holds both)
    constexpr int MO = NP >= 16 ? NP / 16 : 1;  // row tiles of o, the last MO
    // k and alpha (rows) while the paths are walked; then the decayed rows D k and D q,
    // then (D k) S0 and the writes u, with a row's 16-byte quads XORed by its index,
    // so that 16 rows at one column meet distinct banks. (One region for both, where
    // they had two: workgroups a compute unit 2 -> 3 for 32 nodes, 1 -> 2 for 48.)
    __shared__ __attribute__((aligned(16))) float s_buf[2 * NP * D];
    float(*s_k)[D] = reinterpret_cast<float(*)[D]>(s_buf);
    float(*s_al)[D] = s_k + NP;
    auto row = [&](int r, int c) { return &s_buf[r * D + ((((c >> 2) ^ r) & 15) << 2) + (c & 64) + (c & 3)]; };
    // P[i][j] = q_i . D(i,j) k_j at [i][j] (j <= i), A[i][j] = k_i . D(i,j) k_j at [j][i] (j < i)
    __shared__ __attribute__((aligned(16))) float s_pa[NP][LP];
    __shared__ float s_beta[NP];
    __shared__ int s_par[64];
    const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int m16 = lane & 15, q4 = lane >> 4;
    const int N = a.N;

    // load. First what the walk needs, then the state: loads return in order, so
    // the walk waits for the small ones alone and runs while the state arrives.
    // (Places past the end read the last node's rows; unused.)
    typedef Raw<TIN, CT> R;
    typedef Raw<TS, CT> RS;
    constexpr int KR = NP / (2 * NW), WR = (NP + 4 * NW - 1) / (4 * NW);  // rows of k and g a thread, nodes a 16-lane group walks
    const size_t base = ((size_t)b * N * a.H + h) * D;
    auto at = [&](int i) { return (uint32_t)min(i, N - 1) * (uint32_t)(a.H * D); };  // row of node i from `base`
    const TIN* pk = static_cast<const TIN*>(a.k) + base;
    const TIN* pg = static_cast<const TIN*>(a.g) + base;
    const TIN* pq_ = static_cast<const TIN*>(a.q) + base;
    const TIN* pv = static_cast<const TIN*>(a.v) + base;
    const int c2 = CW * wave + CT * m16;  // this lane's CT value channels
    // the n-th node this lane's group of 16 walks: later nodes lie deeper, so the
    // odd rounds deal their nodes the other way about (places past the end as they are)
    auto walk_node = [&](int n) {
        const int first = 4 * NW * n, x = 4 * wave + q4, count = min(4 * NW, N - first);
        return first + (n % 2 && x < count ? count - 1 - x : x);
    };
    const int parent_in = load_parent(a.parents + (size_t)b * N, N);
    typename R::R4 rk[KR], rg[KR], rq[WR][2];
    typename R::RC rv[MO][4];
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        const uint32_t o = at((t >> 5) + 2 * NW * r) + 4 * (t & 31);
        rk[r] = *reinterpret_cast<const typename R::R4*>(pk + o);
        rg[r] = *reinterpret_cast<const typename R::R4*>(pg + o);
    }
#pragma unroll
    for (int r = 0; r < WR; ++r)
#pragma unroll
        for (int p = 0; p < 2; ++p)
            rq[r][p] = *reinterpret_cast<const typename R::R4*>(pq_ + at(walk_node(r)) + 64 * p + 4 * m16);
#pragma unroll
    for (int m = 0; m < MO; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) rv[m][e] = *reinterpret_cast<const typename R::RC*>(pv + at(16 * m + 4 * q4 + e) + c2);
    const float beta = ld(static_cast<const TIN*>(a.beta) + ((size_t)b * N + min(t, N - 1)) * a.H + h);
    asm volatile("" ::: "memory");
    // element s of group g is row 16 g + 4 q4 + s, columns c2 .. (streamed once; a
    // uniform base, a 32-bit lane offset and constants: one address register)
    const TS* S = static_cast<const TS*>(a.state) + (size_t)bh * D * D + CW * wave;
    const uint32_t s_off = 4 * q4 * D + CT * m16;
    typename RS::RC raw[8][4];
#pragma unroll
    for (int g = 0; g < 8; ++g)
#pragma unroll
        for (int s = 0; s < 4; ++s) 
            raw[g][s] = __builtin_nontemporal_load(reinterpret_cast<const typename RS::RC*>(S + 16 * g * D + (s_off + s * D)));
    asm volatile("" ::: "memory");

    const int parent = tree_parent(parent_in);
    const uint64_t there = __ballot(parent != -2);  // lanes past N hold -2
    auto row_of = [&](int i) { return ((size_t)b * N + i) * a.H + h; };
    if (wave == 0) s_par[lane] = parent;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        const int i = (t >> 5) + 2 * NW * r, c = 4 * (t & 31);
        f32x4 g = R::f4(rg[r]);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = __expf(fmaxf(g[e], a.lower_bound));
        *reinterpret_cast<f32x4*>(&s_k[i][c]) = R::f4(rk[r]);
        *reinterpret_cast<f32x4*>(&s_al[i][c]) = g;
    }
    if (t < NP) s_beta[t] = beta;
    for (int e = t; e < NP * LP; e += 64 * NW) (&s_pa[0][0])[e] = 0.0f;
    lds_barrier();

    // walk: node i by 16 lanes, lane channels 4 m16 .. and 64 + 4 m16 ..
    f32x4 kd[WR][2], qd[WR][2];  // the decayed rows wait here until everyone has walked
#pragma unroll
    for (int n = 0; n < WR; ++n) {
        const int i = walk_node(n);
        if (i >= NP) break;
        int j = there >> i & 1 ? i : -1;
        f32x4 q[2], k[2], decay[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            q[p] = k[p] = f32x4{0.f, 0.f, 0.f, 0.f};
            decay[p] = f32x4{1.f, 1.f, 1.f, 1.f};
            if (j >= 0) {
                q[p] = R::f4(rq[n][p]);
                k[p] = *reinterpret_cast<const f32x4*>(&s_k[i][64 * p + 4 * m16]);
            }
        }
        // kAhead: k and alpha of the next node up are read while this one's products run
        f32x4 kj[2] = {k[0], k[1]}, al[2];
        auto read_al = [&](int n) {
#pragma unroll
            for (int p = 0; p < 2; ++p) al[p] = *reinterpret_cast<const f32x4*>(&s_al[n][64 * p + 4 * m16]);
        };
        auto read_k = [&](int n, f32x4* to) {
#pragma unroll
            for (int p = 0; p < 2; ++p) to[p] = *reinterpret_cast<const f32x4*>(&s_k[n][64 * p + 4 * m16]);
        };
        int up = j;
        if (j >= 0) {
            up = s_par[j];
            if constexpr (kAhead) read_al(j);
        }
        while (j >= 0) {
            const int next = max(up, 0), up2 = s_par[next];
            f32x4 kn[2], an[2];
            if constexpr (kAhead) {
                read_k(next, kn);
#pragma unroll
                for (int p = 0; p < 2; ++p) an[p] = *reinterpret_cast<const f32x4*>(&s_al[next][64 * p + 4 * m16]);
            } else {
                read_k(j, kj);
                read_al(j);
            }
            float pq = 0.0f, pk = 0.0f;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                kj[p] *= decay[p];
                decay[p] *= al[p];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pq += q[p][e] * kj[p][e];
                    pk += k[p][e] * kj[p][e];
                }
            }
            pq = sum16(pq);
            pk = sum16(pk);
            if (m16 == 0) {
                s_pa[i][j] = pq;
                if (j != i) s_pa[j][i] = pk;
            }
            j = up;
            up = up2;
            if constexpr (kAhead) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    kj[p] = kn[p];
                    al[p] = an[p];
                }
            }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            kd[n][p] = k[p] * decay[p];
            qd[n][p] = q[p] * decay[p];
        }
    }
    lds_barrier();
#pragma unroll
    for (int n = 0; n < WR; ++n) {
        const int i = walk_node(n);
        if (i >= NP) break;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            *reinterpret_cast<f32x4*>(row(i, 64 * p + 4 * m16)) = kd[n][p];
            *reinterpret_cast<f32x4*>(row(NP + i, 64 * p + 4 * m16)) = qd[n][p];
        }
    }
    lds_barrier();

    // the products' accumulators: rows 4 q4 + e of a tile, columns c2 ...
    // The tiles of (D k) S0 start at -v, so that they end at minus the
    // substitution's right-hand side.
    f32x4 acc[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cols v = 0.0f;
            if (m < MO && (NP >= 16 || q4 < 2)) v = R::fc(rv[m][e]);
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[m][c][e] = -v[c];
        }

    // read: lane (m16, q4) gives row m16 of a tile, K element 16 g + 4 q4 + s in
    // step (g, s), and takes rows 4 q4 + e of column tile c (columns CT m16 + c)
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        f32x4 x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = *reinterpret_cast<const f32x4*>(row(16 * m + m16, 16 * g + 4 * q4));
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const cols st = RS::fc(raw[g][s]);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[m][s], st[c], acc[m][c], 0, 0, 0);
        }
    }
    lds_barrier();  // the rows are read: they now take (D k) S0 and u, each wavefront its own columns
    __builtin_amdgcn_sched_barrier(0);

    // solve: the 64 / CW lanes of a channel hold the same values
    const int col = CW * wave + (lane & (CW - 1));
    // An infinite or NaN write must reach the nodes below it and no others, but
    // the sums below run over all nodes with coefficients 0 where there is no
    // path. So such a write enters the sums as 0, and is noted: it and what lies
    // below it become NaN at the end. (No branch in here: the compiler would sink
    // the updates past it, to where their r is used, and keep every A alive.)
    uint64_t bad = 0;
    static_for<MO>([&](auto I) {
        // the blocks before: (D k) S0 - v + A u on the accumulators
        static_for<I>([&](auto J) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = 16 * J + 4 * q4 + s;
                const float A = s_pa[k][16 * I + m16];
                const cols u = *reinterpret_cast<const cols*>(row(NP + k, c2));
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[I][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(A, u[c], acc[I][c], 0, 0, 0);
            }
        });
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (NP >= 16 || q4 < 2) {
                cols v;
#pragma unroll
                for (int c = 0; c < CT; ++c) v[c] = acc[I][c][e];
                *reinterpret_cast<cols*>(row(16 * I + 4 * q4 + e, c2)) = v;
            }
        wave_lds_order();  // (the wavefront's own columns: its other lanes' rows)
        // within the block
        constexpr int BN_ = NP < 16 ? NP : 16, i0 = 16 * I;
        float r[BN_], beta_[BN_];
        static_for<BN_>([&](auto n) {
            r[n] = -*row(i0 + n, col);
            beta_[n] = s_beta[i0 + n];
        });
        // row j of A is read while row j - 1 is used
        f32x4 A[2][BN_ / 4];
        auto read_A = [&](auto J) {
            static_for<BN_ / 4>([&](auto n) {
                if constexpr (4 * n + 3 > J) A[J % 2][n] = *reinterpret_cast<const f32x4*>(&s_pa[i0 + J][i0 + 4 * n]);
            });
        };
        read_A(std::integral_constant<int, 0>{});
        static_for<BN_>([&](auto J) {
            constexpr int j = J;
            if constexpr (j + 1 < BN_) read_A(std::integral_constant<int, j + 1>{});
            const float u = there >> (i0 + j) & 1 ? beta_[j] * r[j] : 0.0f;
            const bool fine = fabsf(u) < __builtin_inff();
            const float w = fine ? u : 0.0f;
            if (!fine) bad |= (uint64_t)1 << (i0 + j);
            *row(NP + i0 + j, col) = w;
            static_for<BN_>([&](auto n) {
                if constexpr (n > j) r[n] -= A[j % 2][n / 4][n % 4] * w;
            });
            __builtin_amdgcn_sched_barrier(0);  // keep the reads ahead, and no further
        });
        wave_lds_order();  // u of the block, for the blocks after, the writes and o
        __builtin_amdgcn_sched_barrier(0);
    });
    const bool any_bad = __any(bad != 0);
    if (a.writes) {
        constexpr int kLanes = CW / 4;  // of a row
        const int cw = CW * wave + 4 * (lane % kLanes);
#pragma unroll
        for (int i0 = 0; i0 < NP; i0 += 64 / kLanes) {
            const int i = i0 + lane / kLanes;
            if (i < N)
                __builtin_nontemporal_store(*reinterpret_cast<const f32x4*>(row(NP + i, cw)),
                                            reinterpret_cast<f32x4*>(a.writes + row_of(i) * D + cw));
        }
    }
    // o: the last MO row tiles hold (D q) S0; add P u
#pragma unroll
    for (int g = 0; g < (NP + 15) / 16; ++g) {
        cols u[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = 16 * g + 4 * q4 + s;
            u[s] = 0.0f;
            if (NP >= 16 || k < NP) u[s] = *reinterpret_cast<const cols*>(row(NP + (NP >= 16 ? k : k & 7), c2));
        }
#pragma unroll
        for (int m = g; m < MO; ++m) {
            const int i = NP >= 16 ? 16 * m + m16 : m16 - 8;  // the node of this lane's row
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = 16 * g + 4 * q4 + s;
                const float p = k <= i ? s_pa[NP >= 16 ? i : i & 7][NP >= 16 ? k : k & 7] : 0.0f;
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    acc[MT - MO + m][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(p, u[s][c], acc[MT - MO + m][c], 0, 0, 0);
            }
        }
    }
    TOUT* o = static_cast<TOUT*>(a.o);
#pragma unroll
    for (int m = 0; m < MO; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = (NP >= 16 ? 16 * m : -8) + 4 * q4 + e;
            if (i < 0 || i >= N) continue;
            cols v;
#pragma unroll
            for (int c = 0; c < CT; ++c) v[c] = there >> i & 1 ? a.scale * acc[MT - MO + m][c][e] : 0.0f;
            TOUT* p = o + row_of(i) * D + c2;
            if constexpr (sizeof(TOUT) == 4) *reinterpret_cast<cols*>(p) = v;
            else if constexpr (CT == 2) *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
            else st(p, v[0]);
        }
    if (any_bad) {
        // rare: NaN for every write that is not finite and for what lies below it
        asm volatile("" ::: "memory");  // over the stores above, which other lanes made:
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        asm volatile("" ::: "memory");
        for (int i = 0; i < N; ++i) {
            uint64_t above = 0;
            for (int j = __builtin_amdgcn_readlane(parent, i); j >= 0; j = __builtin_amdgcn_readlane(parent, j))
                above |= (uint64_t)1 << j;
            if (!(there >> i & 1) || lane >= CW) continue;
            if (!(bad & (above | (uint64_t)1 << i))) continue;
            if (a.writes) a.writes[row_of(i) * D + col] = __builtin_nanf("");
            st(o + row_of(i) * D + col, __builtin_nanf(""));
        }
    }
}

// ------------------------------------------------------------ commit
// S <- Diag(D(i)) S + sum_j (D(i, j) k_j) u_j^T over the accepted path, in place:
// one read and one write of the state. Threads and columns as the decode step:
// 16 bytes of state per thread and row. The path's decayed keys are formed 16
// nodes at a time, from the accepted node up.
template <typename TS> struct CommitMap {
    static constexpr int kCols = 16 / (int)sizeof(TS);
    static constexpr int kThreads = tree_commit_threads(sizeof(TS) == 4 ? F32 : BF16);
    static constexpr int kLanesPerRow = D / kCols;
    static constexpr int kRowGroups = kThreads / kLanesPerRow;
    static constexpr int kRows = D / kRowGroups;
};
constexpr int kPathChunk = 16;

template <typename TIN, typename TS>
__global__ __launch_bounds__(CommitMap<TS>::kThreads) void tree_commit_kernel(TreeArgs a)
{
    using M = CommitMap<TS>;
    constexpr int kCols = M::kCols, kRows = M::kRows;
    __shared__ __attribute__((aligned(16))) float s_w[kPathChunk][D];
    __shared__ float s_decay[D];
    const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const int N = a.N, t = threadIdx.x;
    const int parent = tree_parent(load_parent(a.parents + (size_t)b * N, N));
    const int acc = a.accepted[b];
    if (acc < 0 || acc >= N || __builtin_amdgcn_readlane(parent, acc & 63) == -2) return;  // uniform over the workgroup
    const int c0 = kCols * (t % M::kLanesPerRow), rg = t / M::kLanesPerRow;
    TS* S = static_cast<TS*>(a.state_out) + (size_t)bh * D * D;
    u32x4_t raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        raw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(S + (size_t)(rg + M::kRowGroups * i) * D + c0));
    float add[kRows][kCols];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int e = 0; e < kCols; ++e) add[i][e] = 0.0f;
    float decay = 1.0f;  // threads 0 .. 127: channel t, from the accepted node up to here
    for (int j0 = acc; j0 >= 0;) {
        int j = j0, n = 0;
        for (; n < kPathChunk && j >= 0; ++n, j = __builtin_amdgcn_readlane(parent, j))
            if (t < D) {
                const size_t row = (((size_t)b * N + j) * a.H + h) * D + t;
                s_w[n][t] = ld(static_cast<const TIN*>(a.k) + row) * decay;
                decay *= __expf(fmaxf(ld(static_cast<const TIN*>(a.g) + row), a.lower_bound));
            }
        if (j < 0 && t < D) s_decay[t] = decay;
        __syncthreads();
        j = j0;
        for (int p = 0; p < n; ++p, j = __builtin_amdgcn_readlane(parent, j)) {
            float u[kCols];
            const float* pu = a.writes_in + (((size_t)b * N + j) * a.H + h) * D + c0;
#pragma unroll
            for (int e = 0; e < kCols; e += 4) *reinterpret_cast<f32x4*>(u + e) = *reinterpret_cast<const f32x4*>(pu + e);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float w = s_w[p][rg + M::kRowGroups * i];
#pragma unroll
                for (int e = 0; e < kCols; ++e) add[i][e] += w * u[e];
            }
        }
        j0 = j;
        if (j0 >= 0) __syncthreads();  // s_w is read
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = rg + M::kRowGroups * i;
        float s[kCols];
        Vec16<TS>::unpack(raw[i], s);
#pragma unroll
        for (int e = 0; e < kCols; ++e) s[e] = s_decay[r] * s[e] + add[i][e];
        __builtin_nontemporal_store(Vec16<TS>::pack(s), reinterpret_cast<u32x4_t*>(S + (size_t)r * D + c0));
    }
}

template <typename TIN, typename TOUT, typename TS>
hipError_t launch_tree_t(const TreeArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((int64_t)a.B * a.H)), block(256), wide(512);
    if (a.N <= 8) hipLaunchKernelGGL((decode_tree_kernel<TIN, TOUT, TS, 8>), grid, block, 0, s, a);
    else if (a.N <= 16) hipLaunchKernelGGL((decode_tree_kernel<TIN, TOUT, TS, 16>), grid, block, 0, s, a);
    else if (a.N <= 32) hipLaunchKernelGGL((decode_tree_kernel<TIN, TOUT, TS, 32>), grid, block, 0, s, a);
    else if (a.N <= 48) hipLaunchKernelGGL((decode_tree_kernel<TIN, TOUT, TS, 48>), grid, wide, 0, s, a);
    else hipLaunchKernelGGL((decode_tree_kernel<TIN, TOUT, TS, 64>), grid, wide, 0, s, a);
    return hipGetLastError();
}
template <typename TIN>
hipError_t launch_tree_in(const TreeArgs& a, hipStream_t s)
{
    if (a.state_dtype == F32)
        return a.out_dtype == F32 ? launch_tree_t<TIN, float, float>(a, s) : launch_tree_t<TIN, bf16_t, float>(a, s);
    return a.out_dtype == F32 ? launch_tree_t<TIN, float, bf16_t>(a, s) : launch_tree_t<TIN, bf16_t, bf16_t>(a, s);
}

template <typename T, int W>
hipError_t launch_conv_w(const ConvTreeArgs& a, hipStream_t s)
{
    if (a.accepted) {
        hipLaunchKernelGGL((conv_commit_kernel<T, W>), dim3((unsigned)a.B, (unsigned)((a.C + 2047) / 2048)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    // LDS for 24 rows serves the usual trees several workgroups at a time, for 72 any
    const dim3 grid((unsigned)a.B, (unsigned)((a.C + 511) / 512));
    if (a.N + W - 1 <= 24) hipLaunchKernelGGL((conv_tree_kernel<T, W, 24>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((conv_tree_kernel<T, W, 72>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_conv_t(const ConvTreeArgs& a, hipStream_t s)
{
    switch (a.W) {
        case 2: return launch_conv_w<T, 2>(a, s);
        case 3: return launch_conv_w<T, 3>(a, s);
        case 4: return launch_conv_w<T, 4>(a, s);
        case 5: return launch_conv_w<T, 5>(a, s);
        case 6: return launch_conv_w<T, 6>(a, s);
        case 7: return launch_conv_w<T, 7>(a, s);
        case 8: return launch_conv_w<T, 8>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_decode_tree(const TreeArgs& a, hipStream_t s)
{
    return a.in_dtype == F32 ? launch_tree_in<float>(a, s) : launch_tree_in<bf16_t>(a, s);
}

hipError_t launch_tree_commit(const TreeArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((int64_t)a.B * a.H));
    if (a.state_dtype == F32) {
        const dim3 block(CommitMap<float>::kThreads);
        if (a.in_dtype == F32) hipLaunchKernelGGL((tree_commit_kernel<float, float>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((tree_commit_kernel<bf16_t, float>), grid, block, 0, s, a);
    } else {
        const dim3 block(CommitMap<bf16_t>::kThreads);
        if (a.in_dtype == F32) hipLaunchKernelGGL((tree_commit_kernel<float, bf16_t>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((tree_commit_kernel<bf16_t, bf16_t>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_conv_tree(const ConvTreeArgs& a, hipStream_t s)
{
    return a.dtype == F32 ? launch_conv_t<float>(a, s) : launch_conv_t<bf16_t>(a, s);
}

}  // namespace kda
