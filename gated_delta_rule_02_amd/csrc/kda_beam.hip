// kda_beam.hip -- beam search: the best continuations of every sequence's beams, and
// the recurrent states that follow them (gfx950).
//
// Selection. A beam w of score S_w offers every token v at
//   c[w, v] = S_w + x[w, v] - log sum_u exp(x[w, u]);
// an ended one offers its end token alone, at S_w. The W best of the W V offers,
// equal ones by lower beam, then lower token, are the new beams.
//
// Bound by HBM: one read of the logits. A wavefront runs along a part of a row
// with the running maximum and sum of the softmax in each lane and the part's W best
// values in order across its lanes (value and token, lane i the i-th): a step of
// 1024 logits costs one comparison of the lanes' maxima with the W-th best, and only
// steps that hold a better value look at their elements. The first step starts from
// the W-th largest of the lanes' maxima (its upper 16 bits, found by bisection
// with ballots), a bound that at least W values reach. A second kernel joins the
// parts, and the beams in 64 bits: beams are compared by sums of scores whose
// rounding to 32 bits would make new ties.
#include <algorithm>

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {
namespace {

// ---------------------------------------------------------------- ordered lists
// float32 bits in the order of the values (as unsigned; 0 stands for "none"); -0 and 0
// are one value
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// the value of the lane before (lane 0: 0), by the wavefront shift of the vector unit: a
// list's shifts follow one another, and a shuffle through LDS takes many times as long
__device__ __forceinline__ uint32_t lane_before(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x138, 0xf, 0xf, false);
}

__device__ __forceinline__ bool finite(float f) { return fabsf(f) < __builtin_inff(); }

// The W best of what was put in, lane i the i-th: higher key first, then lower index.
struct BestList {
    uint32_t key = 0, index = 0xffffffffu;
    __device__ __forceinline__ void put(uint32_t k, uint32_t i, int lane)
    {
        // lanes whose entry comes before the new one form a prefix
        const int pos = __popcll(__ballot(key > k || (key == k && index < i)));
        const uint32_t pk = lane_before(key), pi = lane_before(index);
        if (lane > pos) key = pk, index = pi;
        if (lane == pos) key = k, index = i;
    }
    // every lane's (k, i) with `in` set
    __device__ __forceinline__ void put_lanes(bool in, uint32_t k, uint32_t i, int lane)
    {
        uint64_t todo = __ballot(in);
        while (todo) {
            const int from = __ffsll((unsigned long long)todo) - 1;
            todo &= todo - 1;
            put((uint32_t)__builtin_amdgcn_readlane((int)k, from), (uint32_t)__builtin_amdgcn_readlane((int)i, from), lane);
        }
    }
    __device__ __forceinline__ uint32_t key_of(int place) const { return (uint32_t)__builtin_amdgcn_readlane((int)key, place); }
};

// a bound that at least n of the lanes' keys reach: the n-th largest, its lower 16 bits
// cleared (1, below every key, if fewer lanes have a key)
__device__ __forceinline__ uint32_t lower_bound_of(uint32_t k, int n)
{
    uint32_t bound = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t t = bound | (1u << bit);
        if (__popcll(__ballot(k >= t)) >= n) bound = t;
    }
    return bound | (bound == 0);
}

// ---------------------------------------------------------------- first pass
constexpr int kStep = 1024;  // logits of a wavefront's step: 16 a lane

// 16 values of a step, v of 16 bytes at a time; the row may start anywhere (its
// length may be odd), so these are unaligned loads
template <typename T>
__device__ __forceinline__ void load_step(const T* row, int at, int end, int lane, float* x)
{
    constexpr int VEC = Vec16<T>::N;
    if (at + kStep <= end) {
#pragma unroll
        for (int j = 0; j < 16 / VEC; ++j) {
            u32x4_t u;
            __builtin_memcpy(&u, row + at + (j * 64 + lane) * VEC, 16);
            Vec16<T>::unpack(u, x + j * VEC);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = at + (i / VEC * 64 + lane) * VEC + i % VEC;
            x[i] = e < end ? ld(row + e) : -__builtin_inff();
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void beam_part_kernel(BeamSelectArgs a)
{
    constexpr int VEC = Vec16<T>::N;
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (unit >= (int64_t)a.B * a.W * a.parts) return;
    const int64_t row_i = unit / a.parts;
    const int part = unit % a.parts;
    const T* row = static_cast<const T*>(a.logits) + row_i * a.ld;
    const int begin = part * a.part_len, end = min(begin + a.part_len, a.V);
    float x[16];
    load_step(row, begin, end, lane, x);
    // an ended or dead beam's logits decide nothing
    if ((a.finished && a.finished[row_i]) || !finite(a.scores[row_i])) return;

    float top = -3.402823466e38f, sum = 0.0f;  // finite, so that -inf - top is no NaN
    BestList best;
    uint32_t bound = 0;  // keys below it cannot be among the W best
    for (int at = begin; at < end; at += kStep) {
        if (at != begin) load_step(row, at, end, lane, x);
        float here = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) here = fmaxf(here, x[i]);
        const float m = fmaxf(top, here);
        sum *= exp2_fast((top - m) * kLog2e);
        top = m;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += exp2_fast((x[i] - m) * kLog2e);
        const uint32_t k = at + lane * VEC < end ? order_key(here) : 0;
        if (at == begin) bound = lower_bound_of(k, a.W);
        if (!__ballot(k >= bound)) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = at + (i / VEC * 64 + lane) * VEC + i % VEC;
            const uint32_t ki = order_key(x[i]);
            best.put_lanes(e < end && ki >= bound, ki, (uint32_t)e, lane);
            bound = max(bound, best.key_of(a.W - 1));  // (one as large may be of a lower token: in this step)
        }
        const uint32_t last = best.key_of(a.W - 1);
        if (last) bound = max(bound, last + 1);  // later ones have higher tokens
    }
    // join the lanes
    const float m = wave_max(top);
    double s = (double)(sum * exp2_fast((top - m) * kLog2e));
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
    if (lane == 0) {
        a.part_top[unit] = m;
        a.part_sum[unit] = s;
    }
    if (lane < a.W) {
        a.part_key[unit * a.W + lane] = best.key;
        a.part_token[unit * a.W + lane] = best.index;
    }
}

// ---------------------------------------------------------------- second pass
// A workgroup per sequence. A wavefront joins the parts of a beam: its sum, and of the
// entries that reach the W-th largest of the parts' best the W first. Then
// every offer finds its place: its own in its beam's list and, by bisection, how many
// of every other beam's list come before it.
constexpr int kMaxW = 32;

__global__ __launch_bounds__(1024) void beam_join_kernel(BeamSelectArgs a)
{
    __shared__ double value[kMaxW][kMaxW];
    __shared__ uint32_t token[kMaxW][kMaxW];
    __shared__ uint8_t ended[kMaxW];
    const int lane = threadIdx.x & 63, W = a.W, entries = a.parts * W;
    const int64_t b = blockIdx.x;
    const double none = -__builtin_inf();
    for (int w = threadIdx.x >> 6; w < W; w += blockDim.x >> 6) {
        const int64_t row = b * W + w;
        const uint32_t *keys = a.part_key + row * entries, *tokens = a.part_token + row * entries;
        // lane p: part p (what an ended or dead beam's parts hold is not used)
        const bool on = lane < a.parts;
        const float top = on ? a.part_top[row * a.parts + lane] : -3.402823466e38f;
        const double sum = on ? a.part_sum[row * a.parts + lane] : 0.0;
        const uint32_t head = on ? keys[lane * W] : 0;
        const bool done = a.finished && a.finished[row];
        const float score = a.scores[row];
        const bool dead = !finite(score);
        double v = none;
        uint32_t t = lane;  // a dead beam offers its first tokens, at -inf
        if (!done && !dead) {
            const float m = wave_max(top);
            double s = sum * exp((double)top - (double)m);
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
            if (s > 0.0 && s < __builtin_inf()) {  // not so if no logit is finite, or one is +inf or NaN: dead
                BestList best;
                uint32_t bound = lower_bound_of(head, W);
                for (int e = 0; e < entries; e += 256) {
                    uint32_t k[4], i[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = e + j * 64 + lane;
                        k[j] = at < entries ? keys[at] : 0;
                        i[j] = at < entries ? tokens[at] : 0;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        best.put_lanes(k[j] >= bound, k[j], i[j], lane);
                        bound = max(bound, best.key_of(W - 1));
                    }
                }
                t = best.index;
                if (best.key) v = (double)score + ((double)key_value(best.key) - (double)m - log(s));
            }
        } else if (!dead) {
            // ended: its end token at its score, then the first others at -inf
            if (lane == 0) t = (uint32_t)a.eos, v = (double)score;
            else t = lane - 1 < a.eos ? lane - 1 : lane;
        }
        if (lane < W) {
            value[w][lane] = v;
            token[w][lane] = t;
        }
        if (lane == 0) ended[w] = done;
    }
    __syncthreads();
    const int n = min(W, a.V);  // offers of a beam
    for (int i = threadIdx.x; i < W * n; i += blockDim.x) {
        const int w = i / n, j = i % n;
        const double v = value[w][j];
        int place = j;
        for (int u = 0; u < W && place < W; ++u) {
            if (u == w) continue;
            // the entries of beam u before this one: larger, or equal and of a lower beam
            int lo = 0, hi = n;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                const double o = value[u][mid];
                if (o > v || (o == v && u < w)) lo = mid + 1;
                else hi = mid;
            }
            place += lo;
        }
        if (place < W) {
            const int64_t o = b * W + place;
            const int32_t t = (int32_t)token[w][j];
            a.next_scores[o] = (float)v;
            a.parents[o] = w;
            a.tokens[o] = t;
            if (a.next_finished) a.next_finished[o] = ended[w] || t == a.eos;
        }
    }
}

// ---------------------------------------------------------------- states
// Rows of a sequence's W beams exchanged in place: a thread owns the same 16 bytes
// of every beam, loads those that another beam takes over, then stores them. Only
// beams that another one follows are read and only beams that change are written.
template <int MAXW>
__global__ __launch_bounds__(256) void beam_reorder_kernel(BeamReorderArgs a)
{
    const int64_t state_blocks = (a.state_vecs + 255) / 256, conv_blocks = (a.conv_vecs + 255) / 256;
    const int64_t per = state_blocks + a.streams * conv_blocks;
    for (int64_t blk = blockIdx.x; blk < per * a.B; blk += gridDim.x) {
        const int64_t b = blk / per, i = blk % per;
        int64_t vecs, at;
        u32x4_t* base;
        if (i < state_blocks) {
            vecs = a.state_vecs, at = i * 256 + threadIdx.x;
            base = static_cast<u32x4_t*>(a.state) + b * a.W * vecs;
        } else {
            const int64_t j = i - state_blocks;
            vecs = a.conv_vecs, at = j % conv_blocks * 256 + threadIdx.x;
            base = static_cast<u32x4_t*>(a.conv) + (j / conv_blocks * a.B + b) * a.W * vecs;
        }
        // followers[p]: the beams (but p) that become p's continuation
        uint32_t followers[MAXW];
#pragma unroll
        for (int p = 0; p < MAXW; ++p) followers[p] = 0;
        for (int w = 0; w < a.W; ++w) {
            const int from = a.parents[b * a.W + w];
#pragma unroll
            for (int p = 0; p < MAXW; ++p)
                if (p == from && p < a.W && p != w) followers[p] |= 1u << w;
        }
        if (at >= vecs) continue;
        u32x4_t v[MAXW];
#pragma unroll
        for (int p = 0; p < MAXW; ++p)
            if (followers[p]) v[p] = base[p * vecs + at];
#pragma unroll
        for (int p = 0; p < MAXW; ++p)
            for (uint32_t f = followers[p]; f; f &= f - 1) base[(int64_t)(__ffs(f) - 1) * vecs + at] = v[p];
    }
}

}  // namespace

int beam_part_count(int64_t rows, int64_t V, int* len)
{
    // enough wavefronts to fill the chip (16 a compute unit), whole steps, at most a
    // part for every lane of the joining wavefront
    const int64_t steps = (V + kStep - 1) / kStep;
    const int64_t want = std::min<int64_t>(64, std::max<int64_t>(1, 4096 / rows));
    const int64_t per = (steps + want - 1) / want;
    *len = (int)(per * kStep);
    return (int)((steps + per - 1) / per);
}

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t s)
{
    const int64_t units = (int64_t)a.B * a.W * a.parts;
    const dim3 grid((unsigned)((units + 3) / 4));
    if (a.dtype == F32) hipLaunchKernelGGL((beam_part_kernel<float>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((beam_part_kernel<bf16_t>), grid, dim3(256), 0, s, a);
    hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)a.B), dim3(64 * std::min(a.W, 16)), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const BeamReorderArgs& a, hipStream_t s)
{
    const int64_t per = (a.state_vecs + 255) / 256 + a.streams * ((a.conv_vecs + 255) / 256);
    const dim3 grid((unsigned)min(per * a.B, (int64_t)1 << 20)), block(256);
    if (a.W <= 4) hipLaunchKernelGGL((beam_reorder_kernel<4>), grid, block, 0, s, a);
    else if (a.W <= 8) hipLaunchKernelGGL((beam_reorder_kernel<8>), grid, block, 0, s, a);
    else if (a.W <= 16) hipLaunchKernelGGL((beam_reorder_kernel<16>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((beam_reorder_kernel<32>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
