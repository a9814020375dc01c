// ep_router.hip -- the router in front of the dispatch: the choice of K
// experts per token with their weights, the balance loss with the experts'
// counts, and one backward kernel for both.
//
// Scores.  z is a row of logits; a NaN or +inf logit counts as masked, like
// -inf: it is never chosen and its score is 0.  softmax: s_e = exp(z_e - m),
// m = max z.  sigmoid: s_e = 1 / (1 + exp(-z_e)); where every z_e of the sum
// lies below kSmallSigmoid, exp(z_e - m) stands for it, which differs from
// s_e / s_m by less than 2^-28 and does not underflow.
//
// Everything here is one wave per row: a row's logits are read once into
// registers, and sums and maxima are reductions over the 64 lanes.  Shared memory
// holds the choice's histogram and candidates, a block's column sums and counts for
// the loss, and the scatter of the backward.
#include "ep_common.h"
#include "ep_internal.h"

namespace ep {

namespace {


template <int V>
struct vpl_t {
    static constexpr int value = V;
};
constexpr float kSmallSigmoid = -20.0f;

// Between a write to shared memory and another lane's read of it, and back: the
// lanes of a wave run together and the LDS takes their accesses in order, so this
// only keeps the compiler from moving them across.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------- a row
// A logit as fp32; invalid ones (NaN, +inf) give -inf and are flagged.  The
// addition of +0 turns -0 into +0, so that the two are one value in the order.
struct F32 {
    typedef float type;
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
    typedef float f2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ void get2(const float *p, float &a, float &b)
    {
        const f2 v = *reinterpret_cast<const f2 *>(p);
        a = v[0];
        b = v[1];
    }
    static __device__ __forceinline__ void put2(float *p, float a, float b)
    {
        *reinterpret_cast<f2 *>(p) = f2{a, b};
    }
};
struct Bf16 {
    typedef uint16_t type;
    static __device__ __forceinline__ float get(const uint16_t *p) { return bf16_lo(*p); }
    static __device__ __forceinline__ void put(uint16_t *p, float v)
    {
        *p = (uint16_t)pack_bf16_any(v, v);
    }
    static __device__ __forceinline__ void get2(const uint16_t *p, float &a, float &b)
    {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
        a = bf16_lo(v);
        b = bf16_hi(v);
    }
    static __device__ __forceinline__ void put2(uint16_t *p, float a, float b)
    {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16_any(a, b);
    }
};
__device__ __forceinline__ bool bad_logit(float z)
{
    return !(z < __builtin_huge_valf());
}
__device__ __forceinline__ float clean_logit(float z)
{
    return bad_logit(z) ? kNegInf : z + 0.0f;
}

// exp(x) for x <= 0, to 4u (u = 2^-24) of its value, 0 below 2^-126: 2^t with
// t = x log2(e) as a rounded product and what it lost, and log2(e) in two parts.
// 7 instructions, one of them v_exp_f32, where the library's expf takes about twice
// as many for arguments and results that do not occur here.
__device__ __forceinline__ float exp_f(float x)
{
    constexpr float hi = 1.44269502f, lo = 1.92596299e-8f, ln2 = 0.693147182f;
    x = fmaxf(x, -200.0f);          // -inf too
    const float t = x * hi;
    const float rest = fmaf(x, lo, fmaf(x, hi, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    return fmaf(p, rest * ln2, p);
}
// 1 / (1 + exp(-z)), to 8u of its value (v_rcp_f32: 2u), and 1 minus that.
__device__ __forceinline__ float sigmoid_f(float z)
{
    const float e = exp_f(-fabsf(z));
    return (z < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
}
__device__ __forceinline__ float one_minus_sigmoid_f(float z) { return sigmoid_f(-z); }

// Order-preserving bits: larger float, larger integer; 0 is below them all
// and stands for a masked entry.
__device__ __forceinline__ uint32_t order_bits(float v)
{
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// How a wave's lanes share a row where the order does not matter: value j of a
// lane is expert at(j).  In pairs (E even: rows keep their alignment), a lane's
// loads and stores take two neighbours at once.
template <typename L, int VPL, bool PAIR>
struct Row {
    static_assert(!PAIR || VPL % 2 == 0, "whole pairs");
    static __device__ __forceinline__ int at(int j, int lane)
    {
        return PAIR ? (j >> 1) * (2 * kWave) + lane * 2 + (j & 1) : j * kWave + lane;
    }
    static __device__ __forceinline__ void load(const typename L::type *row, int E, int lane,
                                                float (&z)[VPL])
    {
#pragma unroll
        for (int j = 0; j < VPL; j += PAIR ? 2 : 1) {
            const int e = at(j, lane);
            if constexpr (PAIR) {
                z[j] = z[j + 1] = kNegInf;
                if (e < E)
                    L::get2(row + e, z[j], z[j + 1]);
            } else {
                z[j] = e < E ? L::get(row + e) : kNegInf;
            }
        }
    }
    static __device__ __forceinline__ void store(typename L::type *row, int E, int lane,
                                                 const float (&d)[VPL])
    {
#pragma unroll
        for (int j = 0; j < VPL; j += PAIR ? 2 : 1) {
            const int e = at(j, lane);
            if (e >= E)
                continue;
            if constexpr (PAIR)
                L::put2(row + e, d[j], d[j + 1]);
            else
                L::put(row + e, d[j]);
        }
    }
};

// Row scores for the probabilities: see the head of the file.  `top` is the
// row's maximum (-inf in a row that is masked throughout).
__device__ __forceinline__ float row_score(float z, float top, bool sigmoid)
{
    if (!(z > kNegInf))
        return 0.0f;
    return sigmoid && top >= kSmallSigmoid ? sigmoid_f(z) : exp_f(z - top);
}

// ---------------------------------------------------------------- the choice
// The order of two keys sigmoid(z) + bias that lie this close (relative to
// max(1, |key|)) is not settled in fp32.  With u = 2^-24: v_exp_f32 of
// -z log2(e) and v_rcp_f32 are off by 2u of their values, the product by u of
// its own; as |z| sigmoid'(z) <= 0.3 that makes a score off by less than 4u,
// and the addition of the bias by u of the key.  Two keys: below 10u < 2^-20.
constexpr float kKeyGap = 0x1p-20f;
constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float key_sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}
__device__ __forceinline__ bool finite_f(float v) { return fabsf(v) < __builtin_huge_valf(); }
__device__ __forceinline__ double lane_value_d(double v, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double exact_key(float z, float bias)
{
    return 1.0 / (1.0 + exp(-(double)z)) + (double)bias;
}

// The choice by sigmoid(z) + bias in fp64 over the row in memory: K rounds,
// each taking the first entry after the last one in the order (key descending,
// index ascending).  Only for rows with more than 64 candidates.
template <typename L>
__device__ void choose_fp64(const typename L::type *row, const float *bias, int E, int K, int lane,
                            int &my_e, float &my_z, int &rank)
{
    double last_d = __builtin_huge_val();
    int last_e = -1;
    my_e = -1;
    my_z = kNegInf;
    rank = lane;
    for (int k = 0; k < K; ++k) {
        double best = -__builtin_huge_val();
        int be = 0x7FFFFFFF;
        for (int e = lane; e < E; e += kWave) {
            const float z = clean_logit(L::get(row + e));
            if (!(z > kNegInf) || !finite_f(key_sigmoid(z) + bias[e]))
                continue;
            const double d = exact_key(z, bias[e]);
            if (!(d < last_d || (d == last_d && e > last_e)))
                continue;
            if (be == 0x7FFFFFFF || d > best) {
                best = d;
                be = e;
            }
        }
        for (int m = 1; m < kWave; m <<= 1) {
            const double od = __shfl_xor(best, m);
            const int oe = __shfl_xor(be, m);
            if (oe != 0x7FFFFFFF && (be == 0x7FFFFFFF || od > best || (od == best && oe < be))) {
                best = od;
                be = oe;
            }
        }
        if (be == 0x7FFFFFFF)
            return;
        if (lane == k) {
            my_e = be;
            my_z = clean_logit(L::get(row + be));
        }
        last_d = best;
        last_e = be;
    }
}

// One wave per token.  The keys are the logits (both scores are monotone in
// them, so without a bias the order is exact), or sigmoid(z) + bias.
//
// Candidates: a histogram of the keys over 64 equal steps between the largest
// key and a key that at least K reach (the least of the lanes' best ones) gives
// the step that the K-th falls into; everything from that step up, K and a few
// more, goes to one lane each through shared memory, in index order.  The step
// of a key is monotone in it, whatever the rounding, so nothing below can be
// among the K.  Each candidate then counts those before it.  Rows with more
// than 64 candidates (many equal keys, or a huge range) bisect the border
// between the K and the rest instead, with ballots.
// At 16384 x 384 in bf16, K = 16: K maxima over the wave, one after the other,
// took 43.5 us; bisecting the border in every row 27 us; this 16.5 us, of which 3 to 4
// are the launch and the rest the issue of 465 vector and 158 scalar instructions a
// row (the rows' 13 MB are 3 us).  4096 x 256, K = 8, sigmoid and bias: 6.4 us.
template <typename L, int VPL>
__global__ void __launch_bounds__(256)
route_kernel(const typename L::type *__restrict__ logits, int T, int E, int K, int sigmoid,
             const float *__restrict__ bias, int renorm, float scale,
             int32_t *__restrict__ topk_idx, float *__restrict__ topk_w,
             int32_t *__restrict__ num_invalid)
{
    // the upper half of both takes what has no place, a slot per lane: cheaper
    // than a branch per value
    __shared__ u32x2 chosen[4][2 * kWave];      // expert, logit
    __shared__ int steps[4][2 * kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int nowhere = kWave + lane;
    const int nw = gridDim.x * (blockDim.x / kWave);
    constexpr float kInf = __builtin_huge_valf();
    for (int64_t t = blockIdx.x * (blockDim.x / kWave) + wave; t < T; t += nw) {
        const typename L::type *row = logits + t * E;
        float z[VPL], key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = j * kWave + lane;
            z[j] = e < E ? L::get(row + e) : kNegInf;
        }
        int bad = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const bool wrong = bad_logit(z[j]);
            bad += wrong;
            z[j] = wrong ? kNegInf : z[j];
            key[j] = z[j];
        }
        if (num_invalid) {
            bad = ballot(bad != 0) ? wave_sum(bad) : 0;
            if (lane == 0)
                num_invalid[t] = bad;
        }
        if (bias) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int e = j * kWave + lane;
                const float v = z[j] > kNegInf ? key_sigmoid(z[j]) + bias[e] : kNegInf;
                key[j] = finite_f(v) ? v : kNegInf;
            }
        }
        // the largest key; the least of the lanes' best, which `want` keys reach
        // if as many lanes have one, else the least key of all
        float best = kNegInf, worst = kInf;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            best = fmaxf(best, key[j]);
            worst = fminf(worst, j * kWave + lane < E ? key[j] : kInf);
        }
        int able = E;
        if (ballot(worst == kNegInf)) {         // some are masked
            able = 0;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                able += __popcll(ballot(key[j] > kNegInf));
        }
        const int want = able < K ? able : K;
        const float top = wave_max_f(best);
        float floor_key = best > kNegInf ? best : kInf;
        if (__popcll(ballot(best > kNegInf)) < want) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                floor_key = fminf(floor_key, key[j] > kNegInf ? key[j] : kInf);
        }
        const float low = -wave_max_f(-floor_key);
        const float per = 63.0f * __builtin_amdgcn_rcpf(top - low);
        // 0 .. 63, monotone; NaN (no range to divide) gives 0, as fmaxf leaves it
        // out; below low and masked: nowhere
        auto step_of = [&](float k) {
            const float b = fminf(fmaxf((k - low) * per, 0.0f), (float)(kWave - 1));
            return k >= low ? (int)b : nowhere;
        };
        int my_e = -1, rank = lane, n = 0;
        float my_z = kNegInf;
        if (want > 0) {
            int at_step[VPL];
            steps[wave][lane] = 0;
            wave_sync();
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                at_step[j] = step_of(key[j]);
                atomicAdd(&steps[wave][at_step[j]], 1);
            }
            wave_sync();
            const int upto = wave_inclusive_scan(steps[wave][kWave - 1 - lane], lane);
            const int at = __ffsll((unsigned long long)ballot(upto >= want)) - 1;
            const int border = kWave - 1 - at;
            n = __builtin_amdgcn_readlane(upto, at);
            // with a bias, also what fp64 might put before the K-th
            const float near_by = bias ? kKeyGap * fmaxf(1.0f, fmaxf(fabsf(top), fabsf(low))) : 0.0f;
            if (bias) {
                n = 0;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    at_step[j] = key[j] > kNegInf ? step_of(key[j] + near_by) : nowhere;
                    n += __popcll(ballot((unsigned)(at_step[j] - border) < (unsigned)(kWave - border)));
                }
            }
            if (n <= kWave) {
                int base = 0;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const bool in = (unsigned)(at_step[j] - border) < (unsigned)(kWave - border);
                    const uint64_t m = ballot(in);
                    const int to = in ? base + lanes_below(m) : nowhere;
                    chosen[wave][to] = u32x2{(uint32_t)(j * kWave + lane), __float_as_uint(z[j])};
                    base += __popcll(m);
                }
            } else if (!bias) {
                // lo: the largest key that `want` keys reach, in order bits; then all
                // greater ones, and the lowest indices among the equal
                uint32_t lo = order_bits(low + 0.0f), hi = order_bits(top + 0.0f) + 1u;
                auto bits = [&](float k) { return k > kNegInf ? order_bits(k + 0.0f) : 0u; };
                while (hi - lo > 1u) {
                    const uint32_t mid = lo + (hi - lo) / 2u;
                    int c = 0;
#pragma unroll
                    for (int j = 0; j < VPL; ++j)
                        c += __popcll(ballot(bits(key[j]) >= mid));
                    if (c >= want)
                        lo = mid;
                    else
                        hi = mid;
                }
                int above = 0, base = 0, equal = 0;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    above += __popcll(ballot(bits(key[j]) > lo));
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const uint32_t k = bits(key[j]);
                    const uint64_t eq = ballot(k == lo);
                    const bool in = k > lo || (k == lo && equal + lanes_below(eq) < want - above);
                    equal += __popcll(eq);
                    const uint64_t m = ballot(in);
                    const int to = in ? base + lanes_below(m) : nowhere;
                    chosen[wave][to] = u32x2{(uint32_t)(j * kWave + lane), __float_as_uint(z[j])};
                    base += __popcll(m);
                }
                n = base;
            }
            wave_sync();
            if (n <= kWave) {
                if (lane < n) {
                    const u32x2 c = chosen[wave][lane];
                    my_e = (int)c[0];
                    my_z = __uint_as_float(c[1]) + 0.0f;
                }
                // the place of each: those with a greater key, or an equal one of a
                // lower index (that is, in a lower lane).  Lanes behind the last
                // candidate hold the least key, so whole fours of them do no harm.
                const int n4 = (n + 3) & ~3;
                rank = 0;
                if (sizeof(typename L::type) == 2 && !bias) {
                    // 16 bits of order, 16 of the index: all different
                    const uint32_t mine = lane < n ? (order_bits(my_z) & 0xFFFF0000u) | (kWave - 1 - lane) : 0u;
                    for (int i = 0; i < n4; i += 4) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            rank += (uint32_t)__builtin_amdgcn_readlane((int)mine, i + q) > mine;
                    }
                } else if (!bias) {
                    for (int i = 0; i < n4; i += 4) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            rank += lane_value(my_z, i + q) > my_z;
                    }
                    // the pairs in order are all there are, unless some are equal
                    if (wave_sum(lane < n ? rank : 0) != n * (n - 1) / 2) {
                        for (int i = 0; i < n; ++i)
                            rank += i < lane && lane_value(my_z, i) == my_z;
                    }
                } else {
                    const float mine = lane < n ? key_sigmoid(my_z) + bias[my_e] : kNegInf;
                    int close = 0;
                    for (int i = 0; i < n; ++i) {
                        const float o = lane_value(mine, i);
                        rank += o > mine;
                        close += fabsf(o - mine) <= near_by;
                    }
                    if (ballot(lane < n && close > 1)) {        // more than itself
                        const double d = lane < n ? exact_key(my_z, bias[my_e]) : -__builtin_huge_val();
                        rank = 0;
                        for (int i = 0; i < n; ++i) {
                            const double o = lane_value_d(d, i);
                            rank += o > d || (o == d && i < lane);
                        }
                    }
                }
                if (lane >= n || rank >= want) {        // no candidate, or not chosen
                    my_e = -1;
                    my_z = kNegInf;
                }
            } else {
                choose_fp64<L>(row, bias, E, K, lane, my_e, my_z, rank);
            }
            wave_sync();
        }

        float w;
        if (!renorm) {
            if (sigmoid) {
                w = my_e >= 0 ? sigmoid_f(my_z) : 0.0f;
            } else {
                // keys are the logits here: top is their maximum
                float total = 0.0f;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    total += row_score(z[j], top, false);
                total = wave_sum_f(total);
                w = my_e >= 0 ? row_score(my_z, top, false) / total : 0.0f;
            }
        } else {
            const float zt = wave_max_f(my_z);
            const float s = row_score(my_z, zt, sigmoid);
            const float sum = wave_sum_f(s);
            w = sum > 0.0f ? s / sum : 0.0f;
        }
        // places without a choice: the lanes behind the chosen, in order
        const uint64_t have = ballot(my_e >= 0);
        const int spare = want + lanes_below(~have);
        const int place = my_e >= 0 ? rank : spare;
        if (place < K) {
            topk_idx[t * K + place] = my_e;
            topk_w[t * K + place] = scale * w;
        }
    }
}

// ---------------------------------------------------------------- the balance loss
// Sequence of token t: the last s with seq[s] <= t (T tokens, seq[S] ends the
// last one); -1 or S outside all of them.
__device__ __forceinline__ int find_sequence(const int32_t *seq, int S, int t)
{
    int lo = 0, hi = S + 1;             // the first index with seq[] > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (seq[mid] > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo - 1;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Partial sums of one chunk of CT tokens: for every sequence s that meets
// chunk c, row c + s of the partials gets the column sums of the
// probabilities, the counts, the live rows and the bad data.  Chunks and
// sequences both run along the tokens, so c + s is another row for every pair
// that meets: nchunk + S rows hold all of them.  A wave sums up to kSumRows of its
// rows in fp32, and those sums, and the waves', in fp64: equal addends round
// the same way each time, so that a sum in fp32 drifts with its length (200 u at
// 2^24 equal rows, u = 2^-24).
//   partial row: E floats (sums), E ints (counts), live, bad index, bad logit
struct BalanceRow {
    float *sum;
    int32_t *count, *live;
};
__device__ __forceinline__ BalanceRow balance_row(float *part, int E, int64_t row)
{
    float *p = part + row * (2 * (int64_t)E + 4);
    int32_t *c = reinterpret_cast<int32_t *>(p + E);
    return {p, c, c + E};
}

constexpr int kSumRows = 64;

// Threads of a block by the row length: a wave keeps E column sums in shared
// memory and 2 VPL values per lane in registers (48 KB at E = 4096, and no
// spills: 16 waves leave 128 registers, 2 leave 512).
constexpr int balance_threads(int vpl) { return vpl <= 8 ? 1024 : (vpl <= 16 ? 512 : 128); }

template <typename L, int VPL, bool PAIR>
__global__ void __launch_bounds__(balance_threads(VPL))
balance_partial_kernel(const typename L::type *__restrict__ logits, int T, int E,
                       const int32_t *__restrict__ topk_idx, int K, int sigmoid,
                       const int32_t *__restrict__ seq, int S, int CT, float *__restrict__ part,
                       unsigned *__restrict__ arrived)
{
    extern __shared__ float lds[];      // [waves][E] sums, then [E] counts, then 3 counters
    const int tid = threadIdx.x, bd = blockDim.x;
    const int lane = tid & (kWave - 1), wave = tid / kWave, nw = bd / kWave;
    int32_t *hist = reinterpret_cast<int32_t *>(lds + (size_t)nw * E);
    int32_t *misc = hist + E;
    if (blockIdx.x == 0 && tid == 0)
        *arrived = 0u;
    const int c = blockIdx.x;
    const int c0 = c * CT, c1 = T - c0 > CT ? c0 + CT : T;
    int s = seq ? clampi(find_sequence(seq, S, c0), 0, S - 1) : 0;
    for (; s < S; ++s) {
        const int q0 = seq ? clampi(seq[s], 0, T) : 0, q1 = seq ? clampi(seq[s + 1], 0, T) : T;
        if (q0 >= c1)
            break;
        const int lo = q0 > c0 ? q0 : c0, hi = q1 < c1 ? q1 : c1;
        if (lo >= hi)
            continue;
        for (int e = tid; e < E + 3; e += bd)
            hist[e] = 0;
        __syncthreads();
        // counts: integer adds, the same in any order
        int bad_i = 0;
        const int64_t i1 = (int64_t)hi * K;
        for (int64_t i = (int64_t)lo * K + tid; i < i1; i += bd) {
            const int e = topk_idx[i];
            if ((unsigned)e < (unsigned)E)
                atomicAdd(&hist[e], 1);
            else
                bad_i += e != -1;
        }
        if (bad_i)
            atomicAdd(&misc[1], bad_i);
        float acc[VPL];
        double sums[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            acc[j] = 0.0f;
            sums[j] = 0.0;
        }
        int live = 0, bad_z = 0;
        // the next row's loads are in flight over a row's sums
        float next[VPL];
        auto load = [&](int64_t t) {
            Row<L, VPL, PAIR>::load(logits + t * E, t < hi ? E : 0, lane, next);
        };
        load((int64_t)lo + wave);
        for (int64_t t = (int64_t)lo + wave; t < hi; t += nw) {
            float z[VPL], top = kNegInf, sum = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                z[j] = next[j];
            load(t + nw);
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                bad_z += bad_logit(z[j]);
                z[j] = clean_logit(z[j]);
                top = fmaxf(top, z[j]);
            }
            top = wave_max_f(top);
            if (!(top > kNegInf))
                continue;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                z[j] = row_score(z[j], top, sigmoid);
                sum += z[j];
            }
            const float inv = __builtin_amdgcn_rcpf(wave_sum_f(sum));
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                acc[j] = fmaf(z[j], inv, acc[j]);
            if (++live % kSumRows == 0) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    sums[j] += (double)acc[j];
                    acc[j] = 0.0f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = Row<L, VPL, PAIR>::at(j, lane);
            if (e < E)
                lds[wave * E + e] = (float)(sums[j] + (double)acc[j]);
        }
        const int bz = wave_sum(bad_z);
        if (lane == 0) {
            atomicAdd(&misc[0], live);
            if (bz)
                atomicAdd(&misc[2], bz);
        }
        __syncthreads();
        const BalanceRow r = balance_row(part, E, (int64_t)c + s);
        for (int e = tid; e < E; e += bd) {
            double v = 0.0;
            for (int w = 0; w < nw; ++w)
                v += (double)lds[w * E + e];
            r.sum[e] = (float)v;
            r.count[e] = hist[e];
        }
        if (tid < 3)
            r.live[tid] = misc[tid];
        __syncthreads();
    }
}

constexpr int kFinalCols = 16, kFinalStrips = 32, kFinalThreads = kFinalCols * kFinalStrips;

// One block per (16 experts, sequence): the sums over the sequence's partial
// rows (in fp64: a sum over all tokens; in a fixed order), the counts, the
// table the backward reads, slope[s][e] = E c_se / (K n_s^2), and the block's
// part of sum_e f_se P_se.  The block that arrives last adds the parts in a
// fixed order: the loss does not depend on which one that is.  It is latency
// that counts here (256 rows of partials, 0.8 MB at E = 384): 32 strips take
// 8 rows each with all their loads in flight; 16 waves of 16 rows, one after
// the other, took 14 us.
__global__ void __launch_bounds__(kFinalThreads)
balance_final_kernel(const float *__restrict__ part, int T, int E, int K,
                     const int32_t *__restrict__ seq, int S, int CT, float coef, int eb,
                     int32_t *__restrict__ counts, float *__restrict__ slope,
                     float *__restrict__ loss, int32_t *__restrict__ num_invalid,
                     double *__restrict__ parts, int32_t *__restrict__ tails,
                     unsigned *__restrict__ arrived)
{
    __shared__ double sums[kFinalStrips][kFinalCols];
    __shared__ int32_t cnts[kFinalStrips][kFinalCols];
    __shared__ int32_t misc[3];
    __shared__ bool last;
    const int tid = threadIdx.x, col = tid % kFinalCols, strip = tid / kFinalCols;
    const int s = blockIdx.x / eb, b = blockIdx.x % eb;
    const int e = b * kFinalCols + col;
    const int q0 = seq ? clampi(seq[s], 0, T) : 0, q1 = seq ? clampi(seq[s + 1], 0, T) : T;
    const int r0 = q0 < q1 ? q0 / CT : 0, r1 = q0 < q1 ? (q1 - 1) / CT + 1 : 0;
    if (tid < 3)
        misc[tid] = 0;
    __syncthreads();
    const int64_t stride = 2 * (int64_t)E + 4;
    const float *p = part + ((int64_t)s + r0) * stride;
    double sum = 0.0;
    int cnt = 0;
    if (e < E) {
#pragma unroll 8
        for (int c = strip; c < r1 - r0; c += kFinalStrips) {
            sum += (double)p[c * stride + e];
            cnt += reinterpret_cast<const int32_t *>(p)[c * stride + E + e];
        }
    }
    for (int i = tid; i < 3 * (r1 - r0); i += kFinalThreads)
        if (const int v = reinterpret_cast<const int32_t *>(p)[i / 3 * stride + 2 * E + i % 3])
            atomicAdd(&misc[i % 3], v);
    sums[strip][col] = sum;
    cnts[strip][col] = cnt;
    __syncthreads();
    for (int half = kFinalStrips / 2; half > 0; half >>= 1) {
        if (strip < half) {
            sums[strip][col] += sums[strip + half][col];
            cnts[strip][col] += cnts[strip + half][col];
        }
        __syncthreads();
    }
    const int n = misc[0];
    if (tid < kWave) {
        double v = 0.0;
        if (tid < kFinalCols && e < E) {
            const double inv = n > 0 ? 1.0 / n : 0.0;
            const double f = (double)E * cnts[0][col] / K * inv;
            counts[(int64_t)s * E + e] = cnts[0][col];
            slope[(int64_t)s * E + e] = (float)(f * inv);
            v = f * sums[0][col] * inv;
        }
        for (int m = kFinalCols / 2; m > 0; m >>= 1)
            v += __shfl_down(v, m);
        if (tid == 0) {
            // agent scope: the last block may run on another XCD
            __hip_atomic_store(&parts[blockIdx.x], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (b == 0)
                for (int i = 0; i < 3; ++i)
                    __hip_atomic_store(&tails[3 * (int64_t)s + i], misc[i], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
            const unsigned before = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_ACQ_REL,
                                                           __HIP_MEMORY_SCOPE_AGENT);
            last = before + 1u == gridDim.x;
        }
    }
    __syncthreads();
    if (!last || tid >= kWave)
        return;
    double all = 0.0;
    int n_live = 0, bad_i = 0, bad_z = 0;
    for (int64_t i = tid; i < (int64_t)S * eb; i += kWave)
        all += __hip_atomic_load(&parts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = tid; i < S; i += kWave) {
        n_live += __hip_atomic_load(&tails[3 * (int64_t)i], __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT) > 0;
        bad_i += __hip_atomic_load(&tails[3 * (int64_t)i + 1], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        bad_z += __hip_atomic_load(&tails[3 * (int64_t)i + 2], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
    }
    for (int m = kWave / 2; m > 0; m >>= 1)
        all += __shfl_down(all, m);
    n_live = wave_sum(n_live);
    bad_i = wave_sum(bad_i);
    bad_z = wave_sum(bad_z);
    if (tid == 0) {
        const double per = n_live > 0 ? 1.0 / n_live : 0.0;
        loss[0] = (float)(coef * all * per);
        slope[(int64_t)S * E] = (float)(coef * per);
        num_invalid[0] = bad_i;
        num_invalid[1] = bad_z;
    }
}

// ---------------------------------------------------------------- the gradient
// d_logits of sum(topk_weights * d_w) + d_loss * loss, one wave per row.
//   weights, renormalised: q_k = w_k / scale, G = scale d_w:
//     d = q_k (G_k - sum_j q_j G_j) [1 - s_k], at the chosen experts only
//   softmax as it is: p_e (G_e - sum_k p_k G_k);  sigmoid as it is: G_k s_k (1 - s_k)
//   balance: g p_e (slope_se - sum_j slope_sj p_j) [1 - s_e],
//     g = d_loss coef / live sequences; zero outside every sequence
// (the factors in brackets for the sigmoid).  The chosen entries' parts meet
// their columns in a row of shared memory; a row of logits is read once, and
// only where probabilities of the whole row are needed.
template <typename L, int VPL, bool PAIR>
__global__ void __launch_bounds__(256)
router_backward_kernel(const typename L::type *__restrict__ logits, int T, int E, int K,
                       int sigmoid, int renorm, float scale, const int32_t *__restrict__ topk_idx,
                       const float *__restrict__ d_w, const float *__restrict__ slope,
                       const int32_t *__restrict__ seq, int S, const float *__restrict__ d_loss,
                       typename L::type *__restrict__ d_logits)
{
    extern __shared__ float lds[];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int nw = gridDim.x * (blockDim.x / kWave);
    float *mine = lds + wave * E;
    const bool dense_w = d_w && !sigmoid && !renorm;
    const bool whole = dense_w || slope;
    const float g = slope ? d_loss[0] * slope[(int64_t)S * E] : 0.0f;
    for (int64_t t = blockIdx.x * (blockDim.x / kWave) + wave; t < T; t += nw) {
        const typename L::type *row = logits + t * E;
        float z[VPL], p[VPL], d[VPL];
        float top = kNegInf, inv = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            d[j] = 0.0f;
        if (whole) {
            Row<L, VPL, PAIR>::load(row, E, lane, z);
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                z[j] = clean_logit(z[j]);
                top = fmaxf(top, z[j]);
            }
            top = wave_max_f(top);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                p[j] = row_score(z[j], top, sigmoid);
                sum += p[j];
            }
            sum = wave_sum_f(sum);
            inv = sum > 0.0f ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                p[j] *= inv;
        }
        if (d_w) {
            int e = -1;
            float G = 0.0f;
            if (lane < K) {
                e = topk_idx[t * K + lane];
                G = scale * d_w[t * K + lane];
            }
            float zk = kNegInf;
            if ((unsigned)e < (unsigned)E)
                zk = clean_logit(L::get(row + e));
            const bool in = zk > kNegInf;
            float v = in ? G : 0.0f;
            if (renorm) {
                const float zt = wave_max_f(zk);
                const float s = row_score(zk, zt, sigmoid);
                const float sum = wave_sum_f(s);
                const float q = sum > 0.0f ? s / sum : 0.0f;
                v = q * (v - wave_sum_f(q * v));
                if (sigmoid && in)
                    v *= one_minus_sigmoid_f(zk);
            } else if (sigmoid && in) {
                v *= sigmoid_f(zk) * one_minus_sigmoid_f(zk);
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int c = Row<L, VPL, PAIR>::at(j, lane);
                if (c < E)
                    mine[c] = 0.0f;
            }
            wave_sync();
            if (in)
                atomicAdd(&mine[e], v);
            wave_sync();
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int c = Row<L, VPL, PAIR>::at(j, lane);
                d[j] = c < E ? mine[c] : 0.0f;
            }
            wave_sync();
            if (dense_w) {
                float dot = 0.0f;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    dot = fmaf(p[j], d[j], dot);
                dot = wave_sum_f(dot);
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    d[j] = p[j] * (d[j] - dot);
            }
        }
        if (slope) {
            const int s = seq ? find_sequence(seq, S, (int)t) : 0;
            if (s >= 0 && s < S) {
                const float *f = slope + (int64_t)s * E;
                float fe[VPL], dot = 0.0f;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const int e = Row<L, VPL, PAIR>::at(j, lane);
                    fe[j] = e < E ? f[e] : 0.0f;
                    dot = fmaf(p[j], fe[j], dot);
                }
                dot = wave_sum_f(dot);
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    float v = g * p[j] * (fe[j] - dot);
                    if (sigmoid && z[j] > kNegInf)
                        v *= one_minus_sigmoid_f(z[j]);
                    d[j] += v;
                }
            }
        }
        Row<L, VPL, PAIR>::store(d_logits + t * E, E, lane, d);
    }
}

// Waves of one row each, at most this many blocks of four; beyond it a wave
// takes several rows.
constexpr int kMaxRowBlocks = 1 << 20;
int row_blocks(int T)
{
    const int64_t b = ((int64_t)T + 3) / 4;
    return b < kMaxRowBlocks ? (int)b : kMaxRowBlocks;
}

// Values per lane for E experts: f(VPL).
template <typename F>
hipError_t with_vpl(int E, F f)
{
    if (E <= 64)
        return f(vpl_t<1>());
    if (E <= 128)
        return f(vpl_t<2>());
    if (E <= 256)
        return f(vpl_t<4>());
    if (E <= 384)
        return f(vpl_t<6>());
    if (E <= 512)
        return f(vpl_t<8>());
    if (E <= 1024)
        return f(vpl_t<16>());
    return f(vpl_t<64>());
}

template <typename L>
hipError_t route_t(const void *logits, int T, int E, int K, bool sigmoid, const float *bias,
                   bool renorm, float scale, int32_t *topk_idx, float *topk_w,
                   int32_t *num_invalid, hipStream_t s)
{
    return with_vpl(E, [&](auto v) {
        route_kernel<L, decltype(v)::value><<<row_blocks(T), 256, 0, s>>>(
            static_cast<const typename L::type *>(logits), T, E, K, sigmoid, bias, renorm, scale,
            topk_idx, topk_w, num_invalid);
        return hipGetLastError();
    });
}

template <typename L>
hipError_t balance_t(const BalancePlan &p, const void *logits, const int32_t *topk_idx, int K,
                     bool sigmoid, const int32_t *seq, float *part, unsigned *arrived,
                     hipStream_t s)
{
    return with_vpl(p.E, [&](auto v) {
        constexpr int threads = balance_threads(decltype(v)::value);
        const size_t lds = ((size_t)(threads / kWave) * p.E + p.E + 3) * 4;
        constexpr int VPL = decltype(v)::value;
        auto *kernel = balance_partial_kernel<L, VPL, false>;
        if constexpr (VPL % 2 == 0)
            if (p.E % 2 == 0)
                kernel = balance_partial_kernel<L, VPL, true>;
        kernel<<<p.nchunk, threads, lds, s>>>(static_cast<const typename L::type *>(logits), p.T, p.E,
                                              topk_idx, K, sigmoid, seq, p.S, p.CT, part, arrived);
        return hipGetLastError();
    });
}

template <typename L>
hipError_t router_backward_t(const void *logits, int T, int E, int K, bool sigmoid, bool renorm,
                             float scale, const int32_t *topk_idx, const float *d_w,
                             const float *slope, const int32_t *seq, int S, const float *d_loss,
                             void *d_logits, hipStream_t s)
{
    return with_vpl(E, [&](auto v) {
        constexpr int VPL = decltype(v)::value;
        auto *kernel = router_backward_kernel<L, VPL, false>;
        if constexpr (VPL % 2 == 0)
            if (E % 2 == 0)
                kernel = router_backward_kernel<L, VPL, true>;
        kernel<<<row_blocks(T), 256, 4 * (size_t)E * sizeof(float), s>>>(
            static_cast<const typename L::type *>(logits), T, E, K, sigmoid, renorm, scale, topk_idx,
            d_w, slope, seq, S, d_loss, static_cast<typename L::type *>(d_logits));
        return hipGetLastError();
    });
}

}  // namespace

BalancePlan make_balance_plan(int T, int E, int S)
{
    BalancePlan p{};
    p.T = T;
    p.E = E;
    p.S = S;
    // up to 256 chunks (one per CU) of at least 16 tokens; T may be next to 2^31
    p.CT = (int)(((int64_t)T + 255) / 256);
    if (p.CT < 16)
        p.CT = 16;
    p.nchunk = T > 0 ? (int)(((int64_t)T + p.CT - 1) / p.CT) : 1;
    p.eb = (E + kFinalCols - 1) / kFinalCols;
    size_t off = 0;
    p.off_arrived = off;
    off = align256(off + 4);
    p.off_part = off;
    off = align256(off + ((size_t)p.nchunk + S) * (2 * (size_t)E + 4) * 4);
    p.off_parts = off;
    off = align256(off + (size_t)S * p.eb * 8);
    p.off_tails = off;
    off = align256(off + (size_t)S * 3 * 4);
    p.bytes = off;
    return p;
}

hipError_t launch_route(const void *logits, bool bf16, int T, int E, int K, bool sigmoid,
                        const float *bias, bool renorm, float scale, int32_t *topk_idx,
                        float *topk_w, int32_t *num_invalid, hipStream_t s)
{
    if (T == 0)
        return hipSuccess;
    return bf16 ? route_t<Bf16>(logits, T, E, K, sigmoid, bias, renorm, scale, topk_idx, topk_w,
                                num_invalid, s)
                : route_t<F32>(logits, T, E, K, sigmoid, bias, renorm, scale, topk_idx, topk_w,
                               num_invalid, s);
}

hipError_t launch_balance(const BalancePlan &p, const void *logits, bool bf16,
                          const int32_t *topk_idx, int K, bool sigmoid, const int32_t *seq,
                          float coef, int32_t *counts, float *slope, float *loss,
                          int32_t *num_invalid, char *ws, hipStream_t s)
{
    float *part = reinterpret_cast<float *>(ws + p.off_part);
    unsigned *arrived = reinterpret_cast<unsigned *>(ws + p.off_arrived);
    hipError_t e = bf16 ? balance_t<Bf16>(p, logits, topk_idx, K, sigmoid, seq, part, arrived, s)
                        : balance_t<F32>(p, logits, topk_idx, K, sigmoid, seq, part, arrived, s);
    if (e != hipSuccess)
        return e;
    balance_final_kernel<<<p.S * p.eb, kFinalThreads, 0, s>>>(
        part, p.T, p.E, K, seq, p.S, p.CT, coef, p.eb, counts, slope, loss, num_invalid,
        reinterpret_cast<double *>(ws + p.off_parts), reinterpret_cast<int32_t *>(ws + p.off_tails),
        arrived);
    return hipGetLastError();
}

hipError_t launch_router_backward(const void *logits, bool bf16, int T, int E, int K, bool sigmoid,
                                  bool renorm, float scale, const int32_t *topk_idx,
                                  const float *d_w, const float *slope, const int32_t *seq, int S,
                                  const float *d_loss, void *d_logits, hipStream_t s)
{
    if (T == 0)
        return hipSuccess;
    return bf16 ? router_backward_t<Bf16>(logits, T, E, K, sigmoid, renorm, scale, topk_idx, d_w,
                                          slope, seq, S, d_loss, d_logits, s)
                : router_backward_t<F32>(logits, T, E, K, sigmoid, renorm, scale, topk_idx, d_w,
                                         slope, seq, S, d_loss, d_logits, s);
}

}  // namespace ep
