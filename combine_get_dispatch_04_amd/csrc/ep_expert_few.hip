// ep_expert_few.hip -- a whole layer of experts for a few tokens (decode), in two
// launches:
//   h[t,e] = silu(Wg_e x_t) * (Wu_e x_t)           e = topk_idx[t, k]
//   out_t  = sum_k w[t,k] Wd_e h[t,e]
// with up = [Wg; Wu] [E, 2I, H] and down = Wd [E, H, I] in bf16 or MXFP4.
//
// Bound by the weights' bytes: every expert that a token names is read once, by
// blocks of 32 weight rows (16 gates and their 16 ups in the first launch) that
// go through all of its tokens.  The n-th named expert's blocks find it
// themselves, from topk_idx; what they found is left for the second launch.
//
// The weight rows are the rows of MFMAs, straight from memory to registers, the
// tokens their columns; a block's waves share the inner dimension and add up in
// LDS.  MXFP4 weights are widened to bf16, which is exact.  x is bf16; h goes
// between the launches as two bf16, a value's nearest and what that left over
// (together within 2^-16 of it), in two sets of columns of one MFMA: half the
// columns that few tokens leave empty.
//
// An expert's part of a token's output goes to memory in fp32; the block that
// arrives last at its columns adds the parts up in the order of k, so that the
// result does not depend on which block that is.
#include "ep_common.h"
#include "ep_internal.h"

namespace ep {

namespace {

constexpr int kRows = 32;               // weight rows of a block
constexpr int kMaxWaves = 8;

// What a lane fetches of its weight rows and columns: bf16.
// acc[f][n]: rows f*16 + (lane >> 4)*4 ..+3 by column n*16 + (lane & 15).
template <bool FP4, int NT>
struct Few {
    f32x4 acc[2][NT];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[f][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // Inner elements [32 s0, 32 s1) of D, in blocks of 32: w[f] and scales[f] are the
    // lane's weight rows, col[n] its columns.
    __device__ __forceinline__ void run(const uint8_t *const (&w)[2], const uint8_t *const (&scales)[2],
                                        const uint16_t *const (&col)[NT], int s0, int s1, int D)
    {
        const int g = (threadIdx.x & (kWave - 1)) >> 4;
        if constexpr (FP4) {
            // four blocks at a time, one per 16 lanes
            constexpr int U = NT <= 2 ? 2 : 1;
            for (int s = s0; s < s1; s += 4 * U) {
                u32x4 c[U][2], x[U][NT][4];
                uint32_t sc[U][2];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int b = s + u * 4 + g;
                    const bool there = b < s1;
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        c[u][f] = there ? ld16_nt(w[f] + (int64_t)b * 16) : u32x4{0u, 0u, 0u, 0u};
                        sc[u][f] = there ? scales[f][b] : 127u;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            x[u][n][q] = there ? ld16(col[n] + b * 32 + q * 8) : u32x4{0u, 0u, 0u, 0u};
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const bf16x8 a = __builtin_bit_cast(bf16x8, e2m1_bf16x8(c[u][f][q], sc[u][f]));
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                acc[f][n] = mfma(a, __builtin_bit_cast(bf16x8, x[u][n][q]), acc[f][n]);
                        }
            }
        } else {
            constexpr int U = NT <= 2 ? 4 : 2;
            for (int s = s0; s < s1; s += U) {
                u32x4 c[U][2], x[U][NT];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = (s + u) * 32 + g * 8;
                    const bool there = s + u < s1 && k < D;
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        c[u][f] = there ? ld16_nt(w[f] + (int64_t)k * 2) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        x[u][n] = there ? ld16(col[n] + k) : u32x4{0u, 0u, 0u, 0u};
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            acc[f][n] = mfma(__builtin_bit_cast(bf16x8, c[u][f]),
                                             __builtin_bit_cast(bf16x8, x[u][n]), acc[f][n]);
            }
        }
    }
    // Every wave's sums to LDS: red[wave][f][n] of 16 x 16, column by column.
    __device__ __forceinline__ void put(float *red)
    {
        const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<f32x4 *>(red + (((wave * 2 + f) * NT + n) * 16 + (lane & 15)) * 16 + (lane >> 4) * 4) =
                    acc[f][n];
    }
};
// Row r of fragment f, column c, summed over the waves.
template <int NT>
__device__ __forceinline__ float added(const float *red, int waves, int f, int c, int r)
{
    float v = 0.0f;
    for (int w = 0; w < waves; ++w)
        v += red[(((w * 2 + f) * NT + (c >> 4)) * 16 + (c & 15)) * 16 + r];
    return v;
}

// A wave's share of the inner blocks.
__device__ __forceinline__ void share(int D, int step, int wave, int waves, int &s0, int &s1)
{
    const int blocks = (D + 31) / 32, steps = (blocks + step - 1) / step;
    s0 = steps * wave / waves * step;
    s1 = least(steps * (wave + 1) / waves * step, blocks);
}

// ---------------------------------------------------------------- the first launch
// The n-th of the experts that topk_idx names, ascending, or -1; their number.
// `bits`: kMaxWords words of shared memory.
constexpr int kMaxWords = 4096 / 32;
__device__ int nth_expert(const FewPlan &p, const int32_t *idx, int n, uint32_t *bits, int *found, int &named, int &bad)
{
    const int tid = threadIdx.x, words = (p.E + 31) / 32;
    for (int i = tid; i < kMaxWords; i += blockDim.x)
        bits[i] = 0u;
    if (tid == 0) {
        found[0] = -1;
        found[2] = 0;
    }
    __syncthreads();
    int wrong = 0;
    for (int i = tid; i < p.T * p.K; i += blockDim.x) {
        const int e = idx[i];
        if ((unsigned)e < (unsigned)p.E)
            atomicOr(&bits[e >> 5], 1u << (e & 31));
        else
            wrong += e != -1;
    }
    if (wrong)
        atomicAdd(&found[2], wrong);
    __syncthreads();
    if (tid < kWave) {              // two words a lane
        const uint32_t b0 = bits[2 * tid], b1 = bits[2 * tid + 1];
        const int c0 = __popc(b0), c1 = __popc(b1);
        const int upto = wave_inclusive_scan(c0 + c1, tid);
        int left = n - (upto - c0 - c1);
        if (left >= 0 && left < c0 + c1 && 2 * tid < words) {
            uint32_t b = left < c0 ? b0 : b1;
            const int base = left < c0 ? 64 * tid : 64 * tid + 32;
            left = left < c0 ? left : left - c0;
            for (; left > 0; --left)
                b &= b - 1u;
            found[0] = base + __ffs(b) - 1;
        }
        if (tid == kWave - 1)
            found[1] = upto;
    }
    __syncthreads();
    named = found[1];
    bad = found[2];
    return found[0];
}

struct Token {
    int entry;          // t * K + the first k that names the expert
    float coef;         // the weights of all that do
};

// The tokens that name expert e, in order.  T <= 128: a token per thread of two
// waves.
__device__ int tokens_of(const FewPlan &p, const int32_t *idx, const float *w, int e, Token *list, int *counts)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    int first = -1;
    float coef = 0.0f;
    if (tid < p.T)
        for (int k = 0; k < p.K; ++k)
            if (idx[tid * p.K + k] == e) {
                coef += w ? w[tid * p.K + k] : 1.0f;
                if (first < 0)
                    first = tid * p.K + k;
            }
    const uint64_t has = ballot(first >= 0);
    if (wave < 2 && lane == 0)
        counts[wave] = __popcll(has);
    __syncthreads();
    if (first >= 0)
        list[(wave ? counts[0] : 0) + lanes_below(has)] = Token{first, coef};
    __syncthreads();
    return counts[0] + counts[1];
}

template <bool FP4, int NT>
__device__ __forceinline__ void up_group(const FewPlan &p, const uint16_t *x, const uint8_t *w, const uint8_t *ws,
                                         int e, int i0, const Token *list, int n, float *red, uint16_t *h)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, waves = blockDim.x / kWave;
    const int row = least(i0 + (lane & 15), p.I - 1);
    const uint8_t *rows[2], *scales[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t r = (int64_t)e * 2 * p.I + f * p.I + row;
        rows[f] = w + r * (FP4 ? p.H / 2 : p.H * 2);
        scales[f] = FP4 ? ws + r * (p.H / 32) : nullptr;
    }
    const uint16_t *col[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c)
        col[c] = x + (int64_t)(list[least(c * 16 + (lane & 15), n - 1)].entry / p.K) * p.H;
    Few<FP4, NT> a;
    a.zero();
    int s0, s1;
    share(p.H, FP4 ? 4 : 1, wave, waves, s0, s1);
    a.run(rows, scales, col, s0, s1, p.H);
    a.put(red);
    __syncthreads();
    for (int i = tid; i < 16 * least(n, 16 * NT); i += blockDim.x) {
        const int c = i >> 4, r = i & 15;
        if (i0 + r >= p.I)
            continue;
        const float gate = added<NT>(red, waves, 0, c, r), up = added<NT>(red, waves, 1, c, r);
        const float v = gate / (1.0f + expf(-gate)) * up;
        const uint32_t hi = pack_bf16_any(v, 0.0f);
        const float rest = v - bf16_lo(hi);
        uint16_t *to = h + (int64_t)list[c].entry * p.I + i0 + r;
        to[0] = (uint16_t)hi;
        // an infinity or a NaN has no rest
        to[p.lower] = (uint16_t)pack_bf16_any(fabsf(rest) < __builtin_huge_valf() ? rest : 0.0f, 0.0f);
    }
    __syncthreads();        // `red` is free
}

template <bool FP4>
__global__ void __launch_bounds__(kMaxWaves *kWave, 4)
few_up_kernel(FewPlan p, const uint16_t *__restrict__ x, const int32_t *__restrict__ idx,
              const float *__restrict__ weights, const uint8_t *__restrict__ w, const uint8_t *__restrict__ ws,
              FewTables t, uint16_t *__restrict__ h, int32_t *__restrict__ num_invalid)
{
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ uint32_t bits[kMaxWords];
    __shared__ int found[3], counts[2];
    __shared__ Token list[kFewTokens];
    const int tid = threadIdx.x;
    const int slices = (p.I + 15) / 16, slice = blockIdx.x % slices, at = blockIdx.x / slices;
    // the second launch's counters
    for (int i = blockIdx.x * blockDim.x + tid; i < p.slices; i += gridDim.x * blockDim.x)
        t.arrived[i] = 0u;
    int named, bad;
    const int e = nth_expert(p, idx, at, bits, found, named, bad);
    if (blockIdx.x == 0 && tid == 0) {
        t.named[0] = named;
        num_invalid[0] = bad;
    }
    if (e < 0)
        return;
    const int n = tokens_of(p, idx, weights, e, list, counts);
    if (slice == 0) {
        if (tid == 0) {
            t.expert[at] = e;
            t.count[at] = n;
        }
        for (int i = tid; i < n; i += blockDim.x) {
            t.entry[at * p.T + i] = list[i].entry;
            t.coef[at * p.T + i] = list[i].coef;
        }
    }
    if (n <= 16)
        up_group<FP4, 1>(p, x, w, ws, e, slice * 16, list, n, red, h);
    else if (n <= 32)
        up_group<FP4, 2>(p, x, w, ws, e, slice * 16, list, n, red, h);
    else
        for (int g = 0; g < n; g += 64)
            up_group<FP4, 4>(p, x, w, ws, e, slice * 16, list + g, n - g, red, h);
}

// ---------------------------------------------------------------- the second launch
// Columns: `half` tokens' nearest bf16, then what those left over.
template <bool FP4, int NT>
__device__ __forceinline__ void down_group(const FewPlan &p, const uint16_t *h, const uint8_t *w, const uint8_t *ws,
                                           int e, int r0, const Token *list, int n, float *red, float *part)
{
    constexpr int half = NT * 8;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, waves = blockDim.x / kWave;
    const uint8_t *rows[2], *scales[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t r = (int64_t)e * p.H + least(r0 + f * 16 + (lane & 15), p.H - 1);
        rows[f] = w + r * (FP4 ? p.I / 2 : p.I * 2);
        scales[f] = FP4 ? ws + r * (p.I / 32) : nullptr;
    }
    const uint16_t *col[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int v = c * 16 + (lane & 15);
        col[c] = h + (int64_t)list[least(v % half, n - 1)].entry * p.I + (v < half ? 0 : p.lower);
    }
    Few<FP4, NT> a;
    a.zero();
    int s0, s1;
    share(p.I, FP4 ? 4 : 1, wave, waves, s0, s1);
    a.run(rows, scales, col, s0, s1, p.I);
    a.put(red);
    __syncthreads();
    for (int i = tid; i < kRows * least(n, half); i += blockDim.x) {
        const int c = i / kRows, r = i % kRows;
        if (r0 + r >= p.H)
            continue;
        const float v = added<NT>(red, waves, r >> 4, c, r & 15) + added<NT>(red, waves, r >> 4, half + c, r & 15);
        // read by a block on any XCD: not left in this one's L2
        __hip_atomic_store(part + (int64_t)list[c].entry * p.H + r0 + r, list[c].coef * v, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
}

template <bool FP4>
__global__ void __launch_bounds__(kMaxWaves *kWave, 4)
few_down_kernel(FewPlan p, const uint16_t *__restrict__ h, const int32_t *__restrict__ idx,
                const uint8_t *__restrict__ w, const uint8_t *__restrict__ ws, FewTables t, float *part,
                uint16_t *__restrict__ out)
{
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ Token list[kFewTokens];
    __shared__ uint64_t firsts[kFewTokens];
    __shared__ bool last;
    const int tid = threadIdx.x, slice = blockIdx.x % p.slices, at = blockIdx.x / p.slices, r0 = slice * kRows;
    const int named = t.named[0];
    if (at >= named && at > 0)
        return;
    if (named > 0) {
        const int e = t.expert[at], n = t.count[at];
        for (int i = tid; i < n; i += blockDim.x)
            list[i] = Token{t.entry[at * p.T + i], t.coef[at * p.T + i]};
        __syncthreads();
        if (n <= 8)
            down_group<FP4, 1>(p, h, w, ws, e, r0, list, n, red, part);
        else if (n <= 16)
            down_group<FP4, 2>(p, h, w, ws, e, r0, list, n, red, part);
        else
            for (int g = 0; g < n; g += 32)
                down_group<FP4, 4>(p, h, w, ws, e, r0, list + g, n - g, red, part);
    }
    // Every wave's parts have arrived where all XCDs see them before the block counts
    // itself, and the last block reads them there: the parts' accesses go past the
    // caches, so that no cache needs writing back or invalidating (which would
    // cost the other blocks what they have there of h).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
        last = named == 0 || __hip_atomic_fetch_add(t.arrived + slice, 1u, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT) == (unsigned)named - 1u;
    __syncthreads();
    if (!last)
        return;
    // each token's entries that stand for an expert: the first one of each
    for (int i = tid; i < p.T; i += blockDim.x) {
        uint64_t m = 0;
        for (int k = 0; k < p.K; ++k) {
            const int e = idx[i * p.K + k];
            bool first = (unsigned)e < (unsigned)p.E;
            for (int o = 0; first && o < k; ++o)
                first = idx[i * p.K + o] != e;
            m |= (uint64_t)first << k;
        }
        firsts[i] = m;
    }
    __syncthreads();
    for (int i = tid; i < p.T * (kRows / 2); i += blockDim.x) {
        const int token = i / (kRows / 2), c = r0 + i % (kRows / 2) * 2;
        if (c >= p.H)
            continue;
        float a = 0.0f, b = 0.0f;
        for (uint64_t m = firsts[token]; m; m &= m - 1) {
            float *from = part + ((int64_t)token * p.K + __ffsll((unsigned long long)m) - 1) * p.H + c;
            a += __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            b += __hip_atomic_load(from + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        *reinterpret_cast<uint32_t *>(out + (int64_t)token * p.H + c) = pack_bf16_any(a, b);
    }
}

__global__ void few_zero_kernel(int32_t *p) { *p = 0; }

int reduce_bytes(int waves) { return waves * 2 * 4 * 256 * 4; }

}  // namespace

FewPlan make_few_plan(int T, int K, int E, int H, int I)
{
    FewPlan p{};
    p.T = T;
    p.K = K;
    p.E = E;
    p.H = H;
    p.I = I;
    p.slices = (H + kRows - 1) / kRows;
    p.most = least(T * K, E);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t entries = (size_t)T * K;
    p.lower = (int64_t)entries * I;
    p.off_arrived = take((size_t)p.slices * 4);
    p.off_named = take(4);
    p.off_expert = take((size_t)p.most * 4);
    p.off_count = take((size_t)p.most * 4);
    p.off_entry = take((size_t)p.most * T * 4);
    p.off_coef = take((size_t)p.most * T * 4);
    p.off_h = take(entries * I * 2 * 2);
    p.off_part = take(entries * H * 4);
    p.bytes = off > 256 ? off : 256;
    return p;
}

hipError_t launch_few(const FewPlan &p, const uint16_t *x, const int32_t *idx, const float *weights, const void *up,
                      const uint8_t *up_scales, const void *down, const uint8_t *down_scales, uint16_t *out,
                      int32_t *num_invalid, char *ws, hipStream_t s)
{
    if (p.T == 0) {
        few_zero_kernel<<<1, 1, 0, s>>>(num_invalid);
        return hipGetLastError();
    }
    FewTables t;
    t.arrived = reinterpret_cast<unsigned *>(ws + p.off_arrived);
    t.named = reinterpret_cast<int32_t *>(ws + p.off_named);
    t.expert = reinterpret_cast<int32_t *>(ws + p.off_expert);
    t.count = reinterpret_cast<int32_t *>(ws + p.off_count);
    t.entry = reinterpret_cast<int32_t *>(ws + p.off_entry);
    t.coef = reinterpret_cast<float *>(ws + p.off_coef);
    uint16_t *h = reinterpret_cast<uint16_t *>(ws + p.off_h);
    float *part = reinterpret_cast<float *>(ws + p.off_part);
    const uint8_t *u = static_cast<const uint8_t *>(up), *d = static_cast<const uint8_t *>(down);
    const int64_t blocks_up = (int64_t)p.most * ((p.I + 15) / 16), blocks_down = (int64_t)p.most * p.slices;
    const int waves = 4;
    const int lds = reduce_bytes(waves);
    if (up_scales) {
        few_up_kernel<true><<<(unsigned)blocks_up, waves * kWave, lds, s>>>(p, x, idx, weights, u, up_scales, t, h, num_invalid);
        few_down_kernel<true><<<(unsigned)blocks_down, waves * kWave, lds, s>>>(p, h, idx, d, down_scales, t, part, out);
    } else {
        few_up_kernel<false><<<(unsigned)blocks_up, waves * kWave, lds, s>>>(p, x, idx, weights, u, nullptr, t, h, num_invalid);
        few_down_kernel<false><<<(unsigned)blocks_down, waves * kWave, lds, s>>>(p, h, idx, d, nullptr, t, part, out);
    }
    return hipGetLastError();
}

}  // namespace ep
