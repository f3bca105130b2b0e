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
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int D = 128;
constexpr int kMaxNodes = 64;  // one lane of a wavefront per node

// The parent of this lane's node: -1 (the state), a node, or -2 (absent, itself
// or through a node above it). Every lane of the wavefront takes part.
__device__ __forceinline__ int tree_parent(const int32_t* parents, int N)
{
    const int lane = threadIdx.x & 63;
    int p = lane < N ? parents[lane] : -2;
    if (p < -1 || p >= lane) p = -2;
    // pointer doubling: after s steps `up` is the 2^s-th node above, or -1 / -2
    int up = p;
#pragma unroll
    for (int s = 0; s < 6; ++s) {
        const int far = __shfl(up, max(up, 0), 64);
        if (up >= 0) up = far;
    }
    return up == -2 ? -2 : p;
}

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

// A lane owns 8 channels, a workgroup 2,048 channels of NB nodes of one
// sequence; the NB x W input rows are all under way before the first is used
// (neighbouring nodes share rows: the caches serve those).
template <typename T, int W, int NB>
__global__ __launch_bounds__(256) void conv_tree_kernel(ConvTreeArgs a)
{
    const int blocks = (a.N + NB - 1) / NB;
    const int b = blockIdx.x / blocks, i0 = (blockIdx.x % blocks) * NB;
    const int parent = tree_parent(a.parents + (size_t)b * a.N, a.N);
    // The lanes hold the tree: none of them may leave before the last readlane
    // (a lane that has left has no value to read). Lanes past C, in a wavefront
    // that has some inside, work on channel 0 and store nothing.
    const int c_own = blockIdx.y * 2048 + 8 * threadIdx.x;
    if (__builtin_amdgcn_readfirstlane(c_own) >= a.C) return;
    const bool in = c_own < a.C;  // C is a multiple of 128: whole 16-lane groups
    const int c = in ? c_own : 0;
    // taps of every node, each lane its own: tap j reads list row tap[j] + W - 1
    int tap[W];
    tap[W - 1] = threadIdx.x & 63;
#pragma unroll
    for (int j = W - 2; j >= 0; --j) tap[j] = step_back(parent, tap[j + 1]);
    const T* x = static_cast<const T*>(a.x) + (size_t)b * a.N * a.x_ld + c;
    const T* hist = static_cast<const T*>(a.hist) + (size_t)b * (W - 1) * a.C + c;
    float win[NB][W][8];
    bool there[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int i = i0 + n;
        there[n] = i < a.N && __builtin_amdgcn_readlane(parent, i < a.N ? i : 0) != -2;
        if (!there[n]) continue;
#pragma unroll
        for (int j = 0; j < W; ++j)
            row8(list_row(x, a.x_ld, hist, a.C, W, __builtin_amdgcn_readlane(tap[j], i)), win[n][j]);
    }
    float w[8 * W], bias[8];
#pragma unroll
    for (int v = 0; v < W; ++v) row8(static_cast<const T*>(a.weight) + (size_t)c * W + 8 * v, w + 8 * v);
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = 0.0f;
    if (a.bias) row8(static_cast<const T*>(a.bias) + c, bias);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        if (i0 + n >= a.N) break;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[e] = there[n] ? bias[e] : 0.0f;
            if (!there[n]) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) acc[e] += w[e * W + j] * win[n][j][e];
            if (a.apply_silu) acc[e] = siluf_(acc[e]);
        }
        if (a.l2_group && there[n]) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += acc[e] * acc[e];
            const float r = rsqrtf(group_sum<16>(ss) + a.l2_eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= r;
        }
        if (in) put8(static_cast<T*>(a.y) + ((size_t)b * a.N + i0 + n) * a.C + c, acc);
    }
}

// hist <- the last W - 1 inputs up to the accepted node (bit copies). A thread
// reads all of its channels' rows before it writes one: in place.
template <typename T, int W>
__global__ __launch_bounds__(256) void conv_commit_kernel(ConvTreeArgs a)
{
    constexpr int NV = 8 * (int)sizeof(T) / 16;
    const int b = blockIdx.x;
    const int parent = tree_parent(a.parents + (size_t)b * a.N, a.N);
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
// One workgroup per (sequence, head), a thread per value channel.
template <typename TIN, typename TOUT, typename TS, int NP>
__global__ __launch_bounds__(128) void decode_tree_kernel(TreeArgs a)
{
    __shared__ float s_k[NP][D], s_al[NP][D], s_kt[NP][D], s_qt[NP][D];  // s_k holds the writes u later
    __shared__ float s_A[NP][NP], s_P[NP][NP];
    const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int N = a.N;
    const int parent = tree_parent(a.parents + (size_t)b * N, N);
    auto at = [&](int i) { return ((size_t)b * N + i) * a.H + h; };  // row of [B, N, H, .]
    for (int i = 0; i < N; ++i) {
        if (__builtin_amdgcn_readlane(parent, i) == -2) continue;
        s_k[i][t] = ld(static_cast<const TIN*>(a.k) + at(i) * D + t);
        s_al[i][t] = __expf(fmaxf(ld(static_cast<const TIN*>(a.g) + at(i) * D + t), a.lower_bound));
    }
    __syncthreads();
    // products of each node with the nodes above it, walking up
    for (int i = wave; i < N; i += 2) {
        if (__builtin_amdgcn_readlane(parent, i) == -2) continue;
        const f32x2 q = ld2(static_cast<const TIN*>(a.q) + at(i) * D + 2 * lane);
        const f32x2 k = ld2(&s_k[i][2 * lane]);
        f32x2 decay = {1.0f, 1.0f};
        for (int j = i; j >= 0; j = __builtin_amdgcn_readlane(parent, j)) {
            const f32x2 kj = ld2(&s_k[j][2 * lane]) * decay;
            const float pq = wave_sum(q.x * kj.x + q.y * kj.y), pk = wave_sum(k.x * kj.x + k.y * kj.y);
            if (lane == 0) {
                s_P[i][j] = pq;
                s_A[i][j] = pk;
            }
            decay *= ld2(&s_al[j][2 * lane]);
        }
        *reinterpret_cast<f32x2*>(&s_kt[i][2 * lane]) = k * decay;
        *reinterpret_cast<f32x2*>(&s_qt[i][2 * lane]) = q * decay;
    }
    __syncthreads();
    const TS* S = static_cast<const TS*>(a.state) + (size_t)bh * D * D + t;
    for (int i0 = 0; i0 < N; i0 += 8) {
        float tk[8], tq[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) tk[n] = tq[n] = 0.0f;
        for (int r = 0; r < D; ++r) {
            const float s = ld(S + (size_t)r * D);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                tk[n] += s_kt[(i0 + n) & (NP - 1)][r] * s;
                tq[n] += s_qt[(i0 + n) & (NP - 1)][r] * s;
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int i = i0 + n;
            if (i >= N) break;
            float u = 0.0f, o = 0.0f;
            if (__builtin_amdgcn_readlane(parent, i) != -2) {
                for (int j = __builtin_amdgcn_readlane(parent, i); j >= 0; j = __builtin_amdgcn_readlane(parent, j)) {
                    u += s_A[i][j] * s_k[j][t];
                    o += s_P[i][j] * s_k[j][t];
                }
                u = ld(static_cast<const TIN*>(a.beta) + at(i)) *
                    (ld(static_cast<const TIN*>(a.v) + at(i) * D + t) - tk[n] - u);
                o = a.scale * (tq[n] + o + s_P[i][i] * u);
                s_k[i][t] = u;
            }
            st(static_cast<TOUT*>(a.o) + at(i) * D + t, o);
            if (a.writes) a.writes[at(i) * D + t] = u;
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
    static constexpr int kThreads = sizeof(TS) == 4 ? 1024 : 256;
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
    const int parent = tree_parent(a.parents + (size_t)b * N, N);
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
    const dim3 grid((unsigned)((int64_t)a.B * a.H)), block(128);
    if (a.N <= 16) hipLaunchKernelGGL((decode_tree_kernel<TIN, TOUT, TS, 16>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((decode_tree_kernel<TIN, TOUT, TS, 64>), grid, block, 0, s, a);
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
    const unsigned cb = (unsigned)((a.C + 2047) / 2048);
    if (a.accepted) {
        hipLaunchKernelGGL((conv_commit_kernel<T, W>), dim3((unsigned)a.B, cb), dim3(256), 0, s, a);
    } else {
        constexpr int NB = W <= 4 && sizeof(T) == 2 ? 4 : 2;
        hipLaunchKernelGGL((conv_tree_kernel<T, W, NB>), dim3((unsigned)((int64_t)a.B * ((a.N + NB - 1) / NB)), cb), dim3(256),
                           0, s, a);
    }
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
