// kda_beam.hip -- beam search: the best continuations of every sequence's beams, and
// the recurrent states that follow them (gfx950).
//
// Selection. A beam w of score S_w offers every token v at
//   c[w, v] = S_w + x[w, v] - log sum_u exp(x[w, u]);
// an ended one offers its end token alone, at S_w. The W best of the W V offers,
// equal ones by lower beam, then lower token, are the new beams.
//
// Bound by HBM, one read of the logits of the beams that have not ended: 64 x 8 beams over 131,072
// float32 logits 66 us, 4.1 TB/s. Small calls by the chain of a step and a joining: 4 beams
// over 32,000 logits 4.5 and 4.9 us in two launches, 8 us in one for 4 over 1000. A wavefront runs along a part of a row
// with the running maximum and sum of the softmax in each lane and the part's W best
// values in order across its lanes (value and token, lane i the i-th): a step of
// 1024 logits costs one comparison of the lanes' maxima with the W-th best, and only
// steps that hold a better value look at their elements. The first step starts from
// the W-th largest of the lanes' maxima (its upper 16 bits, found by bisection
// with ballots), a bound that at least W values reach. Then the parts of a beam are joined,
// and the beams in 64 bits: they are compared by sums of scores whose rounding to 32 bits
// would make new ties.
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

// An entry's place in the order as one number: higher keys first, then lower indexes
// (distinct for distinct indexes; 0 only for none).
__device__ __forceinline__ uint64_t entry(uint32_t key, uint32_t index) { return (uint64_t)key << 32 | (uint32_t)~index; }
__device__ __forceinline__ uint64_t lane_entry(uint64_t e, int lane)
{
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)e, lane);
    return lo | (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(e >> 32), lane) << 32;
}

// The best of what was put in, lane i the i-th.
struct BestList {
    uint64_t e = 0;
    __device__ __forceinline__ void put(uint64_t n, int lane)
    {
        const int pos = __popcll(__ballot(e > n));  // lanes whose entry comes before the new one form a prefix
        const uint64_t before = (uint64_t)lane_before((uint32_t)(e >> 32)) << 32 | lane_before((uint32_t)e);
        e = lane > pos ? before : lane == pos ? n : e;
    }
    // every lane's entry with `in` set
    __device__ __forceinline__ void put_lanes(bool in, uint64_t n, int lane)
    {
        uint64_t todo = __ballot(in);
        while (todo) {
            const int from = __ffsll((unsigned long long)todo) - 1;
            todo &= todo - 1;
            put(lane_entry(n, from), lane);
        }
    }
    // the list of count <= 64 entries, lane i's the i-th (distinct): each counts those before
    // it, which do not wait for one another as puts do (with the rest of that step, 16 beams
    // over 1000 tokens 21 -> 16 us)
    __device__ __forceinline__ void sort(uint64_t n, int count, int lane)
    {
        int rank = lane < count ? 0 : lane;
        for (int c = 0; c < count; ++c) {
            const uint64_t o = lane_entry(n, c);
            rank += lane < count && o > n;
        }
        if (lane >= count) n = 0;
        const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_permute(rank * 4, (int)(uint32_t)n);
        e = (uint64_t)(uint32_t)__builtin_amdgcn_ds_permute(rank * 4, (int)(uint32_t)(n >> 32)) << 32 | lo;
    }
    __device__ __forceinline__ uint32_t key_of(int place) const { return (uint32_t)(lane_entry(e, place) >> 32); }
    __device__ __forceinline__ uint32_t key() const { return (uint32_t)(e >> 32); }
    __device__ __forceinline__ uint32_t index() const { return ~(uint32_t)e; }
};

// Entries picked lane by lane, gathered in LDS (64 of the wavefront's own) to be sorted;
// beyond 64 they only count.
struct Gather {
    uint64_t* slots;
    int count = 0;
    __device__ __forceinline__ void add(bool in, uint64_t n, int lane)
    {
        const uint64_t mask = __ballot(in);
        if (!mask) return;
        const int at = count + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        if (in && at < 64) slots[at] = n;
        count += __popcll(mask);
    }
    __device__ __forceinline__ uint64_t mine(int lane) const
    {
        wave_lds_order();
        const uint64_t n = lane < count ? slots[lane] : 0;
        wave_lds_order();
        return n;
    }
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

// ---------------------------------------------------------------- a wavefront's maximum and sum
// By shifts within rows of 16 lanes and broadcasts of a row's last lane to the next (on the
// vector unit); every lane gets lane 63's.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp<CTRL, ROWS>(0, (uint32_t)u), hi = dpp<CTRL, ROWS>(0, (uint32_t)(u >> 32));
    return __builtin_bit_cast(double, lo | hi << 32);
}
__device__ __forceinline__ float wave_top(float v)
{
    auto step = [&](uint32_t moved) { v = fmaxf(v, __uint_as_float(moved)); };
    step(dpp<0x111, 0xf>(__float_as_uint(v), __float_as_uint(v)));  // from 1, 2, 4 and 8 lanes before
    step(dpp<0x112, 0xf>(__float_as_uint(v), __float_as_uint(v)));
    step(dpp<0x114, 0xf>(__float_as_uint(v), __float_as_uint(v)));
    step(dpp<0x118, 0xf>(__float_as_uint(v), __float_as_uint(v)));
    step(dpp<0x142, 0xa>(__float_as_uint(v), __float_as_uint(v)));  // rows 1 and 3: from the row before
    step(dpp<0x143, 0xc>(__float_as_uint(v), __float_as_uint(v)));  // rows 2 and 3: from row 1
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ double wave_total(double v)
{
    v += dpp_or_zero<0x111, 0xf>(v);
    v += dpp_or_zero<0x112, 0xf>(v);
    v += dpp_or_zero<0x114, 0xf>(v);
    v += dpp_or_zero<0x118, 0xf>(v);
    v += dpp_or_zero<0x142, 0xa>(v);
    v += dpp_or_zero<0x143, 0xc>(v);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, lo | hi << 32);
}

// e^d, d <= 0. log2(e) in two parts that one rounding joins: float32's alone is low by 1.3e-8 of
// it in every term, which put the logarithms of 32,000 logits off by 3.5e-8 on average (this
// way by 0.5e-8, for 1 per cent of the time of 64 x 8 x 131,072 in float32, 3 in bfloat16)
__device__ __forceinline__ float exp_below(float d)
{
    constexpr float kLog2eRest = 1.925963033e-8f;
    return exp2_fast(fmaf(d, kLog2e, d * kLog2eRest));
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

// What the parts of all rows leave for the joining: top (largest logit) and sum (of
// exponentials) per part, and the W best entries.
struct PartResults {
    float* top;
    double* sum;
    uint64_t* entries;
};

// Part `unit` of row `row_i`: the tokens begin .. end - 1.
template <typename T>
__device__ __forceinline__ void part_of_row(const BeamSelectArgs& a, int64_t row_i, int begin, int end, int64_t unit,
                                            const PartResults& out, uint64_t* slots, int lane)
{
    constexpr int VEC = Vec16<T>::N;
    const T* row = static_cast<const T*>(a.logits) + row_i * a.ld;
    float x[16];
    load_step(row, begin, end, lane, x);
    // an ended or dead beam's logits decide nothing
    if ((a.finished && a.finished[row_i]) || !finite(a.scores[row_i])) return;

    float top = -3.402823466e38f;  // finite, so that -inf - top is no NaN
    double sum = 0.0;              // over the steps; a step's own 16 terms in float32
    BestList best;
    uint32_t bound = 0;  // keys below it cannot be among the W best
    for (int at = begin; at < end; at += kStep) {
        if (at != begin) load_step(row, at, end, lane, x);
        float here = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) here = fmaxf(here, x[i]);
        const float m = fmaxf(top, here);
        float part[4] = {};
#pragma unroll
        for (int i = 0; i < 16; ++i) part[i % 4] += exp_below(x[i] - m);
        sum = sum * (double)exp_below(top - m) + (double)((part[0] + part[1]) + (part[2] + part[3]));
        top = m;
        const uint32_t k = at + lane * VEC < end ? order_key(here) : 0;
        if (at == begin) bound = lower_bound_of(k, a.W);
        if (!__ballot(k >= bound)) continue;
        auto token = [&](int i) { return at + (i / VEC * 64 + lane) * VEC + i % VEC; };
        bool sorted = false;
        if (at == begin) {
            Gather g{slots};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t ki = order_key(x[i]);
                g.add(token(i) < end && ki >= bound, entry(ki, (uint32_t)token(i)), lane);
            }
            sorted = g.count <= 64;
            if (sorted) best.sort(g.mine(lane), g.count, lane);
        }
        if (!sorted) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t ki = order_key(x[i]);
                best.put_lanes(token(i) < end && ki >= bound, entry(ki, (uint32_t)token(i)), lane);
                bound = max(bound, best.key_of(a.W - 1));  // (one as large may be of a lower token: in this step)
            }
        }
        const uint32_t last = best.key_of(a.W - 1);
        if (last) bound = max(bound, last + 1);  // later ones have higher tokens
    }
    const float m = wave_top(top);
    const double s = wave_total(sum * (double)exp_below(top - m));
    if (lane == 0) {
        out.top[unit] = m;
        out.sum[unit] = s;
    }
    if (lane < a.W) {
        out.entries[unit * a.W + lane] = best.e;
    }
}

// ---------------------------------------------------------------- joining
// A workgroup joins a sequence, a wavefront a beam's parts: its sum, and of the entries that
// reach a bound the W first. Then every offer finds its place: its own in its beam's list
// and, by bisection, how many of every other beam's list come before it. `in` holds the
// sequence's parts.
constexpr int kMaxW = 32;
struct Offers {
    double value[kMaxW][kMaxW];
    double score[kMaxW], top[kMaxW], log_sum[kMaxW];
    uint32_t token[kMaxW][kMaxW];
    int before[1024];  // of each thread's share of the other beams
    uint8_t ended[kMaxW];
    uint64_t slots[16][64];  // of the wavefronts
};

__device__ __forceinline__ void join_sequence(const BeamSelectArgs& a, int64_t b, const PartResults& in, Offers& offers)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, W = a.W, count = a.parts * W;
    const double none = -__builtin_inf();
    for (int w = wave; w < W; w += blockDim.x >> 6) {
        const int64_t row = b * W + w;
        const uint64_t* entries = in.entries + w * count;
        // lane p: part p (what an ended or dead beam's parts hold is not used)
        const bool on = lane < a.parts;
        const float top = on ? in.top[w * a.parts + lane] : -3.402823466e38f;
        const double sum = on ? in.sum[w * a.parts + lane] : 0.0;
        // and the first entries of every part, as many as there are lanes for: the W-th largest
        // of them is reached by few more than W of all (of the parts' best alone, where the
        // parts are not many more than W, by more than there is room to sort)
        const int of = lane % a.parts, nth = lane / a.parts;
        const uint32_t head = nth < W && nth < 64 / a.parts ? (uint32_t)(entries[of * W + nth] >> 32) : 0;
        uint64_t e[4];  // the first 256, on their way together with the rest
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = j * 64 + lane < count ? entries[j * 64 + lane] : 0;
        const bool done = a.finished && a.finished[row];
        const float score = a.scores[row];
        const bool dead = !finite(score);
        double v = none;
        uint32_t t = lane;  // a dead beam offers its first tokens, at -inf
        bool live = false;
        if (!done && !dead) {
            const float m = a.parts == 1 ? in.top[w] : wave_top(top);
            const double s = a.parts == 1 ? in.sum[w] : wave_total(sum * exp((double)top - (double)m));
            if (s > 0.0 && s < __builtin_inf()) {  // not so if no logit is finite, or one is +inf or NaN: dead
                BestList best;
                if (a.parts == 1) {
                    best.e = e[0];
                } else {
                    const uint32_t bound = lower_bound_of(head, W);
                    Gather g{offers.slots[wave]};
                    for (int at = 0;;) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) g.add((uint32_t)(e[j] >> 32) >= bound, e[j], lane);
                        if ((at += 256) >= count) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j) e[j] = at + j * 64 + lane < count ? entries[at + j * 64 + lane] : 0;
                    }
                    if (g.count <= 64) {
                        best.sort(g.mine(lane), g.count, lane);
                    } else {
                        for (int at = 0; at < count; at += 64) {
                            const uint64_t n = at + lane < count ? entries[at + lane] : 0;
                            best.put_lanes((uint32_t)(n >> 32) >= max(bound, best.key_of(W - 1)), n, lane);
                        }
                    }
                }
                t = best.index();
                if (best.e) v = (double)key_value(best.key());
                live = true;
                if (lane == 0) offers.top[w] = m, offers.log_sum[w] = s;
            }
        } else if (!dead) {
            // ended: its end token at its score, then the first others at -inf
            if (lane == 0) t = (uint32_t)a.eos, v = (double)score;
            else t = lane - 1 < a.eos ? lane - 1 : lane;
        }
        if (lane < W) {
            offers.value[w][lane] = v;
            offers.token[w][lane] = t;
        }
        if (lane == 0) {
            offers.ended[w] = done;
            offers.score[w] = live ? (double)score : none;  // (none: the values are the offers already)
        }
    }
    __syncthreads();
    if (threadIdx.x < W) offers.log_sum[threadIdx.x] = log(offers.log_sum[threadIdx.x]);  // (all beams' at once)
    __syncthreads();
    for (int i = threadIdx.x; i < W * W; i += blockDim.x) {
        const int w = i / W;
        if (offers.score[w] != none)
            offers.value[w][i % W] = offers.score[w] + ((offers.value[w][i % W] - offers.top[w]) - offers.log_sum[w]);
    }
    __syncthreads();
    // An offer's place: its own in its list and, for every other beam, how many of that one's
    // come before it: larger ones, and equal ones of a lower beam. A thread takes an offer and
    // every `share`-th beam.
    const int n = min(W, a.V), offered = W * n;  // of a beam, of all
    const int share = max(min((int)blockDim.x / offered, W), 1);
    for (int i = threadIdx.x; i < offered * share; i += blockDim.x) {
        const int w = i % offered / n, j = i % n;
        const double v = offers.value[w][j];
        int before = 0;
        for (int u = i / offered; u < W; u += share) {
            int c = 0;
            for (int step = 1 << (31 - __clz(n)); step; step >>= 1) {
                const double o = offers.value[u][min(c + step, n) - 1];
                if (c + step <= n && (o > v || (o == v && u < w))) c += step;
            }
            if (u != w) before += c;
        }
        offers.before[i] = before;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < offered; i += blockDim.x) {
        const int w = i / n, j = i % n;
        int place = j;
        for (int q = 0; q < share; ++q) place += offers.before[q * offered + i];
        if (place < W) {
            const int64_t o = b * W + place;
            const int32_t t = (int32_t)offers.token[w][j];
            a.next_scores[o] = (float)offers.value[w][j];
            a.parents[o] = w;
            a.tokens[o] = t;
            if (a.next_finished) a.next_finished[o] = offers.ended[w] || t == a.eos;
        }
    }
}

// ---------------------------------------------------------------- two launches: parts over the chip
template <typename T>
__global__ __launch_bounds__(256) void beam_part_kernel(BeamSelectArgs a)
{
    __shared__ uint64_t slots[4][64];
    const int wave = threadIdx.x >> 6;
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= (int64_t)a.B * a.W * a.parts) return;
    const int begin = (int)(unit % a.parts) * a.part_len;
    part_of_row<T>(a, unit / a.parts, begin, min(begin + a.part_len, a.V), unit,
                   PartResults{a.part_top, a.part_sum, a.part_entries}, slots[wave], threadIdx.x & 63);
}

__global__ __launch_bounds__(1024) void beam_join_kernel(BeamSelectArgs a)
{
    __shared__ Offers offers;
    const int64_t b = blockIdx.x, units = b * a.W * a.parts;
    join_sequence(a, b, PartResults{a.part_top + units, a.part_sum + units, a.part_entries + units * a.W}, offers);
}

// ---------------------------------------------------------------- one launch: a workgroup per sequence
// where its wavefronts have a part of one step each, at most
constexpr int kOneParts = 16;

template <typename T>
__global__ __launch_bounds__(1024) void beam_one_kernel(BeamSelectArgs a)
{
    __shared__ Offers offers;
    __shared__ float top[kOneParts];
    __shared__ double sum[kOneParts];
    __shared__ uint64_t entries[kOneParts * kOneParts];  // (at most as many beams as parts)
    const int64_t b = blockIdx.x;
    const int part = threadIdx.x >> 6;
    const PartResults parts{top, sum, entries};
    if (part < a.W * a.parts) {
        const int begin = part % a.parts * a.part_len;
        part_of_row<T>(a, b * a.W + part / a.parts, begin, min(begin + a.part_len, a.V), part, parts, offers.slots[part],
                       threadIdx.x & 63);
    }
    __syncthreads();
    join_sequence(a, b, parts, offers);
}

// ---------------------------------------------------------------- states
// Rows of a sequence's W beams exchanged in place: a thread owns the same 16 bytes
// of every beam, loads those that another beam takes over, then stores them. Only
// beams that another one follows are read and only beams that change are written.
template <int MAXW, int THREADS>
__global__ __launch_bounds__(THREADS) void beam_reorder_kernel(BeamReorderArgs a)
{
    const int64_t state_blocks = (a.state_vecs + THREADS - 1) / THREADS, conv_blocks = (a.conv_vecs + THREADS - 1) / THREADS;
    const int64_t per = state_blocks + a.streams * conv_blocks;
    const int lane = threadIdx.x & 63;
    for (int64_t blk = blockIdx.x; blk < per * a.B; blk += gridDim.x) {
        const int64_t b = blk / per, i = blk % per;
        int64_t vecs, at;
        u32x4_t* base;
        if (i < state_blocks) {
            vecs = a.state_vecs, at = i * THREADS + threadIdx.x;
            base = static_cast<u32x4_t*>(a.state) + b * a.W * vecs;
        } else {
            const int64_t j = i - state_blocks;
            vecs = a.conv_vecs, at = j % conv_blocks * THREADS + threadIdx.x;
            base = static_cast<u32x4_t*>(a.conv) + (j / conv_blocks * a.B + b) * a.W * vecs;
        }
        // followers[p]: the beams (but p) that become p's continuation
        const int from = lane < a.W ? a.parents[b * a.W + lane] : -1;
        uint32_t followers[MAXW];
#pragma unroll
        for (int p = 0; p < MAXW; ++p) followers[p] = p < a.W ? (uint32_t)__ballot(from == p && lane != p) : 0;
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

template <int MAXW, int THREADS>
hipError_t launch_reorder(const BeamReorderArgs& a, hipStream_t s)
{
    const int64_t per = (a.state_vecs + THREADS - 1) / THREADS + a.streams * ((a.conv_vecs + THREADS - 1) / THREADS);
    hipLaunchKernelGGL((beam_reorder_kernel<MAXW, THREADS>), dim3((unsigned)min(per * a.B, (int64_t)1 << 20)), dim3(THREADS), 0,
                       s, a);
    return hipGetLastError();
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
    const int steps = (a.V + kStep - 1) / kStep;
    if (a.W * steps <= kOneParts) {
        BeamSelectArgs o = a;
        o.parts = steps;
        o.part_len = kStep;
        if (a.dtype == F32) hipLaunchKernelGGL((beam_one_kernel<float>), dim3((unsigned)a.B), dim3(1024), 0, s, o);
        else hipLaunchKernelGGL((beam_one_kernel<bf16_t>), dim3((unsigned)a.B), dim3(1024), 0, s, o);
        return hipGetLastError();
    }
    const int64_t units = (int64_t)a.B * a.W * a.parts;
    const dim3 grid((unsigned)((units + 3) / 4));
    if (a.dtype == F32) hipLaunchKernelGGL((beam_part_kernel<float>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((beam_part_kernel<bf16_t>), grid, dim3(256), 0, s, a);
    hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)a.B), dim3(64 * std::min(a.W, 16)), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const BeamReorderArgs& a, hipStream_t s)
{
    if (a.W <= 4) return launch_reorder<4, 256>(a, s);
    if (a.W <= 8) return launch_reorder<8, 512>(a, s);
    if (a.W <= 16) return launch_reorder<16, 512>(a, s);
    return launch_reorder<32, 512>(a, s);
}

}  // namespace kda
