// ep_expert_few.hip -- a whole layer of experts for a few tokens (decode), in two
// launches:
//   h[t,e] = silu(Wg_e x_t) * (Wu_e x_t)           e = topk_idx[t, k]
//   out_t  = sum_k w[t,k] Wd_e h[t,e]
// with up = [Wg; Wu] [E, 2I, H] and down = Wd [E, H, I] in bf16 or MXFP4.
//
// Bound by the weights' bytes: an expert that a token names is read by blocks of 32 or 128
// weight rows (half of them gates and half their ups in the first launch).  Blocks of 32
// go through its n tokens in ceil(n / 32) passes over the weight in the first launch and
// ceil(n / 16) in the second; of 128 rows there are ceil(n / 64) and ceil(n / 32) blocks, a
// pass each.  The form is chosen by the sizes alone, whatever the tokens name: 128 tokens,
// 1 of 64 experts (bf16, H 4096, I 2048), take 577 us spread evenly, 352 with 96 of them at
// one expert, and 169 with all there, whose 50 MB are then read four and eight times.  The
// n-th named expert's blocks find it themselves, from topk_idx; what they found is left
// for the second launch.
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
//
// Measured, the first launch and the second: one token, 8 of 64 experts (bf16, H 4096,
// I 2048) 50 + 30 us for 403 MB; the same in MXFP4 with H 7168 35 + 25 for 187 MB, where
// a launch's own time, the search for the expert and the first loads are a third of it;
// 32 tokens in bf16 349 + 193 for 3.2 GB (5.8 TB/s); 128 tokens, 2 of 8 experts in MXFP4
// (H = I = 4096) 54 + 66 for 214 MB: a step of 128 channels takes a block 1.6 us, of which
// its matrix work and its reads of LDS are 0.2 each and its 24 vector memory
// instructions, at about 60 cycles, 0.6; the rest is latency (two blocks to a CU), some of
// it a wait for all loads in flight once in four steps (see run_fp4).
#include "ep_common.h"
#include "ep_internal.h"

namespace ep {

namespace {

constexpr int kMaxWaves = 4;

// A block's columns in LDS, if they fit: rows of bf16, 64 bytes apart beyond their
// length so that 16 columns' reads spread over the banks.  For MXFP4 weights the
// pieces of 8 channels lie in the order of their use: of four blocks of 32 their
// first pieces, their second ones, ...  Zeros behind the last channel.
template <bool FP4>
__host__ __device__ __forceinline__ int column_bytes(int D)
{
    return FP4 ? (D + 127) / 128 * 256 + 64 : (D + 31) / 32 * 64 + 64;
}
template <bool FP4>
__device__ __forceinline__ int column_place(int piece)
{
    return FP4 ? piece / 16 * 256 + (piece & 3) * 64 + (piece >> 2 & 3) * 16 : piece * 16;
}
constexpr int kStageBytes = 32 << 10;   // of a block, at most
constexpr int kFrags = 2;

// The waits for columns on their way to LDS count the loads behind them, so the weight's
// loads have to stay behind the columns' and in front of the next ones: nothing else tells
// the compiler so, which sees two kinds of memory.
__device__ __forceinline__ void loads_stay_in_order()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Two fragments of 16 weight rows by NT of 16 columns, from memory or (STAGED) from LDS.
// acc[f][n]: rows f*16 + (lane >> 4)*4 ..+3 by column n*16 + (lane & 15).
template <bool FP4, int NT, bool STAGED>
struct Few {
    f32x4 acc[kFrags][NT];
    const uint8_t *w[kFrags], *scales[kFrags];    // the lane's weight rows
    const uint16_t *col[NT];            // its columns
    uint32_t at[NT];                    // the same in LDS
    const char *lds;

    __device__ __forceinline__ u32x4 column(int n, int piece) const
    {
        if constexpr (STAGED)
            return ld16(lds + at[n] + column_place<FP4>(piece));
        else
            return ld16(col[n] + piece * 8);
    }
    // Inner elements [32 s0, 32 s1) of D, in blocks of 32.  Every wave of a block comes here:
    // staged columns, on their way, are met behind its own first loads.
    __device__ __forceinline__ void run(int s0, int s1, int D)
    {
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[f][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (FP4)
            run_fp4(s0, s1, D / 32);
        else
            run_bf16(s0, s1, D);
    }
    // Four blocks at a time, one per 16 lanes.  The weight comes from memory and is asked
    // for AHEAD steps before its use, the columns from a cache or LDS, one step.  The
    // scales come sixteen at a time (a row's request is 64 bytes whatever it takes of
    // them), four steps ahead, as loads come back in their order.  But they are loaded in
    // one of two ways, so the compiler cannot count what is in flight behind them, and
    // waits for all of it once in four steps.  (One token, 8 of 64 experts, H 7168, I 2048:
    // with 1, 2 and 3 steps ahead 68, 61 and 66 us: registers.  Without staging they do not
    // suffice as it is: of the 128 that four waves on a SIMD have each, pointers mostly lie
    // in scratch, up to 124 bytes a lane.)
    __device__ __forceinline__ void run_fp4(int s0, int s1, int HB)
    {
        constexpr int SLOTS = 4, AHEAD = NT > 1 ? 1 : 2, RING = AHEAD > 1 ? 4 : 2, XS = NT > 1 ? 1 : 2;
        const int g = (threadIdx.x & (kWave - 1)) >> 4, last = s1 - 1;
        u32x4 c[RING][kFrags], x[XS][NT][4], sc[kFrags], next[kFrags];
        // behind the last block: the last one again, its columns as zeros and its scales
        // as 1 (an infinite one times 0 would be a NaN)
        auto load_w = [&](int s, int slot) {
            const int b = least(s + g, last);
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
                c[slot][f] = ld16_nt(w[f] + (int64_t)b * 16);
        };
        auto load_scales = [&](int s) {
#pragma unroll
            for (int f = 0; f < kFrags; ++f) {
                if (s + 16 <= HB) {
                    __builtin_memcpy(&next[f], scales[f] + s, 16);
                } else {        // the lane's own ones
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        next[f][j] = (uint32_t)scales[f][least(s + 4 * j + g, last)] << (8 * g);
                }
            }
        };
        auto load_x = [&](int s, int slot) {
            const int b = STAGED ? s + g : least(s + g, last);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    x[slot][n][q] = column(n, b * 4 + q);
        };
        auto multiply = [&](int s, int j, int xslot) {
            const bool behind = s + g >= s1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8 v[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    v[n] = __builtin_bit_cast(bf16x8, behind ? u32x4{0u, 0u, 0u, 0u} : x[xslot][n][q]);
#pragma unroll
                for (int f = 0; f < kFrags; ++f) {
                    const uint32_t one = behind ? 127u : sc[f][j] >> (8 * g) & 255u;
                    const bf16x8 a = __builtin_bit_cast(bf16x8, e2m1_bf16x8(c[j % RING][f][q], one));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        acc[f][n] = mfma(a, v[n], acc[f][n]);
                }
            }
        };
        if (s0 >= s1) {
            if constexpr (STAGED)
                wait_and_meet<0>();
            return;
        }
        if constexpr (STAGED)
            loads_stay_in_order();
        load_scales(s0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            load_w(s0 + 4 * j, j);
        if constexpr (STAGED) {
            loads_stay_in_order();
            wait_and_meet<AHEAD * kFrags>();         // the loads of the columns came before these
        }
        load_x(s0, 0);
        for (int s = s0; s < s1; s += 4 * SLOTS) {
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
                sc[f] = next[f];
            if (s + 4 * SLOTS < s1)
                load_scales(s + 4 * SLOTS);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int now = s + 4 * j;
                if (now >= s1)
                    break;
                load_w(now + 4 * AHEAD, (j + AHEAD) % RING);
                if constexpr (XS == 2) {
                    if (now + 4 < s1)
                        load_x(now + 4, (j + 1) % 2);
                    multiply(now, j, j % 2);
                } else {
                    multiply(now, j, 0);
                    if (now + 4 < s1)
                        load_x(now + 4, 0);
                }
            }
        }
    }
    __device__ __forceinline__ void run_bf16(int s0, int s1, int D)
    {
        constexpr int U = 4;
        const int g = (threadIdx.x & (kWave - 1)) >> 4;
        u32x4 c[U][kFrags];
        auto load_w = [&](int s) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (s + u) * 32 + g * 8;
#pragma unroll
                for (int f = 0; f < kFrags; ++f)
                    c[u][f] = s + u < s1 && k < D ? ld16_nt(w[f] + (int64_t)k * 2) : u32x4{0u, 0u, 0u, 0u};
            }
        };
        load_w(s0);
        if constexpr (STAGED)
            wait_and_meet<0>();
        for (int s = s0; s < s1; s += U) {
            u32x4 x[U][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool there = s + u < s1 && (STAGED || (s + u) * 32 + g * 8 < D);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    x[u][n] = there ? column(n, (s + u) * 4 + g) : u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int f = 0; f < kFrags; ++f)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        acc[f][n] = mfma(__builtin_bit_cast(bf16x8, c[u][f]), __builtin_bit_cast(bf16x8, x[u][n]),
                                         acc[f][n]);
            if (s + U < s1)
                load_w(s + U);
        }
    }
    // Every wave's sums to LDS: red[wave][f][n] of 16 x 16, column by column.
    __device__ __forceinline__ void put(float *red)
    {
        const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<f32x4 *>(red + (((wave * kFrags + f) * NT + n) * 16 + (lane & 15)) * 16 + (lane >> 4) * 4) =
                    acc[f][n];
    }
};
// Row r of fragment f, column c, summed over the waves.
template <int NT>
__device__ __forceinline__ float added(const float *red, int waves, int f, int c, int r)
{
    float v = 0.0f;
    for (int w = 0; w < waves; ++w)
        v += red[(((w * kFrags + f) * NT + (c >> 4)) * 16 + (c & 15)) * 16 + r];
    return v;
}

// A wave's share of the inner blocks.
__device__ __forceinline__ void share(int D, int step, int wave, int waves, int &s0, int &s1)
{
    const int blocks = (D + 31) / 32, steps = (blocks + step - 1) / step;
    s0 = steps * wave / waves * step;
    s1 = least(steps * (wave + 1) / waves * step, blocks);
}

// Starts the loads of `n` columns into LDS: column i's bf16 lie at element from(i) of
// the array, which has less than 2^31 bytes.
constexpr uint32_t kNowhere = 0x80000000u;
template <bool FP4, typename C>
__device__ __forceinline__ void stage_columns(char *to, const uint16_t *array, int64_t elements, int n, int D, C from)
{
    const rsrc_t r = row_rsrc(array, (int)(elements * 2));
    const int slots = column_bytes<FP4>(D) / 16, all = n * slots;
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (int p0 = wave * kWave; p0 < all; p0 += blockDim.x) {
        const int p = p0 + lane, c = least(p / slots, n - 1), slot = p % slots;
        // column_place's inverse
        const int piece = FP4 ? (slot & ~15) + (slot & 3) * 4 + (slot >> 2 & 3) : slot;
        const bool there = p < all && slot < slots - 4 && piece * 8 < D;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(to + p0 * 16), 16,
                                                 there ? (uint32_t)(from(c) * 2) + piece * 16 : kNowhere, 0, 0, 0);
    }
}
// Whether so many columns of an array can be staged (in whole loads of a wave).
template <bool FP4>
__device__ __forceinline__ bool can_stage(const FewPlan &p, int n, int D, int64_t elements)
{
    return (n * (int64_t)column_bytes<FP4>(D) + 1023) / 1024 * 1024 <= p.stage_bytes && elements < 1 << 30;
}

// ---------------------------------------------------------------- some tokens for each expert
// Where experts have some tokens each, the columns are what the CUs have to take in: a
// block's four waves then share them, by LDS, and take 32 weight rows each through
// the whole inner dimension.  Steps of 128 elements; a step's columns are rows of
// 256 bytes, piece c of column r in slot c ^ (r & 15).  Columns and weight are asked for
// AHEAD steps before their use: seven where the buffers (64 KB, of two blocks on a CU)
// and the registers reach that far, else three (MXFP4: less behind every fourth step, which
// waits for all loads).
template <bool FP4, int NT>
struct Shared {
    static constexpr int SLOTS = FP4 && NT <= 2 ? 8 : 4, AHEAD = SLOTS - 1, bytes = NT * 4096, WL = FP4 ? 1 : 4;
    f32x4 acc[2][NT];
    const uint8_t *w[2], *scales[2];    // the lane's weight rows
    uint32_t col[NT];                   // offset of the column whose piece the lane loads, or kNowhere
    rsrc_t from;
    char *lds;

    __device__ __forceinline__ void run(int D)
    {
        const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int g = lane >> 4, n = (D + 127) / 128, HB = D / 32;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int c = 0; c < NT; ++c)
                acc[f][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        u32x4 c[SLOTS][2][WL], sc[2], next[2];
        // the columns behind the last element are zeros; the weight's elements there have
        // to be finite
        auto load_w = [&](int s, int slot) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                if constexpr (FP4) {
                    c[slot][f][0] = ld16_nt(w[f] + (int64_t)least(s * 4 + g, HB - 1) * 16);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int k = s * 128 + q * 32 + g * 8;
                        c[slot][f][q] = k < D ? ld16_nt(w[f] + (int64_t)k * 2) : u32x4{0u, 0u, 0u, 0u};
                    }
                }
            }
        };
        auto load_scales = [&](int s) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                if (s * 4 + 16 <= HB) {
                    __builtin_memcpy(&next[f], scales[f] + s * 4, 16);
                } else {        // the lane's own ones; 1 behind the last
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int b = (s + j) * 4 + g;
                        next[f][j] = (b < HB ? (uint32_t)scales[f][b] : 127u) << (8 * g);
                    }
                }
            }
        };
        const int piece = (lane & 15) ^ ((wave * 4 + g) & 15);
        auto load_x = [&](int s) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)(lds + s % SLOTS * bytes + (i * 4 + wave) * 1024), 16,
                                                         s * 128 + piece * 8 < D ? col[i] : kNowhere, s * 256, 0, 0);
        };
        auto load_step = [&](int s, int slot) {
            load_x(s);
            loads_stay_in_order();
            load_w(s, slot);
            loads_stay_in_order();
        };
        auto multiply = [&](int s, int j) {
            const char *const tile = lds + s % SLOTS * bytes + (lane & 15) * 256;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8 x[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    x[i] = __builtin_bit_cast(bf16x8, ld16(tile + i * 4096 + (((FP4 ? g * 4 + q : q * 4 + g) ^ (lane & 15)) << 4)));
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    bf16x8 a;
                    if constexpr (FP4)
                        a = __builtin_bit_cast(bf16x8, e2m1_bf16x8(c[j][f][0][q], sc[f][j % 4] >> (8 * g) & 255u));
                    else
                        a = __builtin_bit_cast(bf16x8, c[j][f][q]);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        acc[f][i] = mfma(a, x[i], acc[f][i]);
                }
            }
        };
        if constexpr (FP4)
            load_scales(0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (j < n)
                load_step(j, j);
        for (int s = 0; s < n; s += SLOTS) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int now = s + j;
                if (now >= n)
                    break;
                if (FP4 && j % 4 == 0) {        // four steps ahead, and a wait for all loads, as above
                    sc[0] = next[0];
                    sc[1] = next[1];
                    if (now + 4 < n)
                        load_scales(now + 4);
                }
                // behind a step's columns come its own weight (in bf16 the last step's may be
                // six loads short, for which it is not counted) and AHEAD - 1 steps
                if (now + AHEAD <= n)
                    wait_and_meet<(AHEAD - 1) * (NT + 2 * WL) + (FP4 ? 2 : 0)>();
                else
                    wait_and_meet<0>();
                if (now + AHEAD < n)
                    load_step(now + AHEAD, (j + AHEAD) % SLOTS);
                multiply(now, j);
            }
        }
        __syncthreads();        // the buffers are free
    }
};

// ---------------------------------------------------------------- the first launch
// The n-th of the experts that topk_idx names, ascending, or -1; their number.
// `bits`: kMaxWords words of shared memory; `entries`: the entries' experts and weights
// there, for what comes after (both loads at once: each is a miss).
constexpr int kMaxWords = 4096 / 32;
struct Entry {
    int e;
    float w;
};
__device__ int nth_expert(const FewPlan &p, const int32_t *idx, const float *w, int n, uint32_t *bits, Entry *entries,
                          int *found, int &named, int &bad)
{
    const int tid = threadIdx.x, words = (p.E + 31) / 32;
    for (int i = tid; i < kMaxWords; i += blockDim.x)
        bits[i] = 0u;
    if (tid == 0) {
        found[0] = -1;
        found[2] = 0;
    }
    for (int i = tid; i < p.T * p.K; i += blockDim.x)
        entries[i] = Entry{idx[i], w ? w[i] : 1.0f};
    __syncthreads();
    int wrong = 0;
    for (int i = tid; i < p.T * p.K; i += blockDim.x) {
        const int e = entries[i].e;
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

// The tokens that name expert e, in order.  T <= 128: a token per lane, 64 at a time.
__device__ int tokens_of(const FewPlan &p, const Entry *entries, int e, Token *list, int *counts)
{
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
    Token mine[2];
    uint64_t has[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int part = wave + i * waves, t = part * kWave + lane;
        mine[i] = Token{-1, 0.0f};
        if (part < 2 && t < p.T) {
#pragma unroll 8
            for (int k = p.K - 1; k >= 0; --k) {
                const Entry v = entries[t * p.K + k];
                const bool same = v.e == e;
                mine[i].coef += same ? v.w : 0.0f;
                mine[i].entry = same ? t * p.K + k : mine[i].entry;
            }
        }
        has[i] = ballot(mine[i].entry >= 0);
        if (part < 2 && lane == 0)
            counts[part] = __popcll(has[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (mine[i].entry >= 0)
            list[(wave + i * waves ? counts[0] : 0) + lanes_below(has[i])] = mine[i];
    __syncthreads();
    return counts[0] + counts[1];
}
// Each token's entries that stand for an expert, the first of each, as bits, and the
// number of all: left for the second launch.  `sum`: a word of shared memory.
__device__ void first_entries(const FewPlan &p, const Entry *entries, uint64_t *firsts, int *sum, int32_t *total)
{
    if (threadIdx.x == 0)
        *sum = 0;
    __syncthreads();
    for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
        uint64_t m = 0;
        for (int k = 0; k < p.K; ++k) {
            const int e = entries[t * p.K + k].e;
            bool again = false;
#pragma unroll 8
            for (int o = 0; o < k; ++o)
                again |= entries[t * p.K + o].e == e;
            m |= (uint64_t)((unsigned)e < (unsigned)p.E && !again) << k;
        }
        firsts[t] = m;
        atomicAdd(sum, __popcll(m));
    }
    __syncthreads();
    if (threadIdx.x == 0)
        *total = *sum;
}

// Fragments: the gates of 16 of the I columns from i0 on, then their ups.
template <bool FP4, int NT, bool STAGED>
__device__ __forceinline__ void up_group(const FewPlan &p, const uint16_t *x, const uint8_t *w, const uint8_t *ws,
                                         int e, int i0, const Token *list, int n, float *red, uint16_t *h)
{
    constexpr int cols = kFrags * 8;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, waves = blockDim.x / kWave;
    Few<FP4, NT, STAGED> a;
    a.lds = reinterpret_cast<const char *>(red);
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
        const int row = least(i0 + f % (kFrags / 2) * 16 + (lane & 15), p.I - 1);
        const int64_t r = (int64_t)e * 2 * p.I + f / (kFrags / 2) * p.I + row;
        a.w[f] = w + r * (FP4 ? p.H / 2 : p.H * 2);
        a.scales[f] = FP4 ? ws + r * (p.H / 32) : nullptr;
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int i = least(c * 16 + (lane & 15), n - 1);
        if constexpr (STAGED)
            a.at[c] = i * column_bytes<FP4>(p.H);
        else
            a.col[c] = x + (int64_t)(list[i].entry / p.K) * p.H;
    }
    int s0, s1;
    share(p.H, FP4 ? 4 : 1, wave, waves, s0, s1);
    if constexpr (STAGED) {
        stage_columns<FP4>(reinterpret_cast<char *>(red), x, (int64_t)p.T * p.H, n, p.H,
                           [&](int i) { return (int64_t)(list[i].entry / p.K) * p.H; });
        a.run(s0, s1, p.H);
        __syncthreads();        // `red` is the columns' memory
    } else {
        a.run(s0, s1, p.H);
    }
    a.put(red);
    __syncthreads();
    for (int i = tid; i < cols * least(n, 16 * NT); i += blockDim.x) {
        const int c = i / cols, r = i % cols;
        if (i0 + r >= p.I)
            continue;
        const float gate = added<NT>(red, waves, r >> 4, c, r & 15),
                    up = added<NT>(red, waves, kFrags / 2 + (r >> 4), c, r & 15);
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

// The same with shared columns: a wave's fragments are 16 gates and their ups.
template <bool FP4, int NT>
__device__ __forceinline__ void up_shared(const FewPlan &p, const uint16_t *x, const uint8_t *w, const uint8_t *ws,
                                          int e, int i0, const Token *list, int n, char *lds, uint16_t *h)
{
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    Shared<FP4, NT> a;
    a.lds = lds;
    a.from = row_rsrc(x, p.T * p.H * 2);
    const int row = i0 + wave * 16;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t r = (int64_t)e * 2 * p.I + f * p.I + least(row + (lane & 15), p.I - 1);
        a.w[f] = w + r * (FP4 ? p.H / 2 : p.H * 2);
        a.scales[f] = FP4 ? ws + r * (p.H / 32) : nullptr;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int c = (i * 4 + wave) * 4 + (lane >> 4);
        a.col[i] = c < n ? (uint32_t)(list[least(c, n - 1)].entry / p.K) * p.H * 2 + (((lane & 15) ^ (c & 15)) << 4) : kNowhere;
    }
    a.run(p.H);
    const int at = row + (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int c = i * 16 + (lane & 15);
        if (c >= n || at >= p.I)        // (n may be more than the 16 NT that are these)
            continue;
        float v[4], rest[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float gate = a.acc[0][i][q];
            v[q] = gate / (1.0f + expf(-gate)) * a.acc[1][i][q];
        }
        const u32x2 hi = {pack_bf16_any(v[0], v[1]), pack_bf16_any(v[2], v[3])};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float r = v[q] - (q & 1 ? bf16_hi(hi[q >> 1]) : bf16_lo(hi[q >> 1]));
            rest[q] = fabsf(r) < __builtin_huge_valf() ? r : 0.0f;      // an infinity or a NaN has no rest
        }
        uint16_t *to = h + (int64_t)list[c].entry * p.I + at;
        *reinterpret_cast<u32x2 *>(to) = hi;
        *reinterpret_cast<u32x2 *>(to + p.lower) = u32x2{pack_bf16_any(rest[0], rest[1]), pack_bf16_any(rest[2], rest[3])};
    }
}

template <bool FP4, bool WIDE>
__global__ void __launch_bounds__(kMaxWaves *kWave, WIDE ? 2 : 4)
few_up_kernel(FewPlan p, const uint16_t *__restrict__ x, const int32_t *__restrict__ idx,
              const float *__restrict__ weights, const uint8_t *__restrict__ w, const uint8_t *__restrict__ ws,
              FewTables t, uint16_t *__restrict__ h, int32_t *__restrict__ num_invalid)
{
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ uint32_t bits[kMaxWords];
    __shared__ int found[3], counts[2];
    __shared__ Token list[kFewTokens];
    const int tid = threadIdx.x;
    // tokens go 64 at a time, each lot to a block of its own; the first lots first
    const int slices = p.slices_up, slice = blockIdx.x % slices, i0 = slice * (WIDE ? 64 : 16);
    const int at = blockIdx.x / slices % p.most, lot = WIDE ? blockIdx.x / slices / p.most : 0;
    // the second launch's counters
    for (int i = blockIdx.x * blockDim.x + tid; i < p.slices; i += gridDim.x * blockDim.x)
        t.arrived[i] = 0u;
    int named, bad;
    // (in the memory of the columns, which come later)
    Entry *const entries = reinterpret_cast<Entry *>(red);
    const int e = nth_expert(p, idx, weights, at, bits, entries, found, named, bad);
    if (blockIdx.x == 0 && tid == 0) {
        t.named[0] = named;
        num_invalid[0] = bad;
    }
    if (blockIdx.x == gridDim.x - 1)
        first_entries(p, entries, t.firsts, counts, t.named + 1);
    if (e < 0)
        return;
    const int n = tokens_of(p, entries, e, list, counts);
    if (slice == 0 && lot == 0) {
        if (tid == 0) {
            t.expert[at] = e;
            t.count[at] = n;
        }
        for (int i = tid; i < n; i += blockDim.x) {
            t.entry[at * p.T + i] = list[i].entry;
            t.coef[at * p.T + i] = list[i].coef;
        }
    }
    if constexpr (WIDE) {
        char *const lds = reinterpret_cast<char *>(red);
        const Token *mine = list + lot * 64;
        const int m = n - lot * 64;
        if (m > 32)
            up_shared<FP4, 4>(p, x, w, ws, e, i0, mine, m, lds, h);
        else if (m > 16)
            up_shared<FP4, 2>(p, x, w, ws, e, i0, mine, m, lds, h);
        else if (m > 0)
            up_shared<FP4, 1>(p, x, w, ws, e, i0, mine, m, lds, h);
    } else {
        if (n <= 16 && can_stage<FP4>(p, n, p.H, (int64_t)p.T * p.H))
            up_group<FP4, 1, true>(p, x, w, ws, e, i0, list, n, red, h);
        else if (n <= 16)
            up_group<FP4, 1, false>(p, x, w, ws, e, i0, list, n, red, h);
        else
            for (int g = 0; g < n; g += 32)
                up_group<FP4, 2, false>(p, x, w, ws, e, i0, list + g, n - g, red, h);
    }
}

// ---------------------------------------------------------------- the second launch
// The sum of a product with h's two parts.  An infinite weight gives an infinity or a NaN with
// the first one; what it gives with the second (a NaN, where nothing was left over, or an
// infinity of the other sign) is not part of the result.
__device__ __forceinline__ float joined(float nearest, float rest)
{
    return fabsf(nearest) < __builtin_huge_valf() ? nearest + rest : nearest;
}

// Columns: `half` tokens' nearest bf16, then what those left over.
template <bool FP4, int NT, bool STAGED>
__device__ __forceinline__ void down_group(const FewPlan &p, const uint16_t *h, const uint8_t *w, const uint8_t *ws,
                                           int e, int r0, const Token *list, int n, float *red, float *part)
{
    constexpr int half = NT * 8, cols = kFrags * 16;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, waves = blockDim.x / kWave;
    Few<FP4, NT, STAGED> a;
    a.lds = reinterpret_cast<const char *>(red);
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
        const int64_t r = (int64_t)e * p.H + least(r0 + f * 16 + (lane & 15), p.H - 1);
        a.w[f] = w + r * (FP4 ? p.I / 2 : p.I * 2);
        a.scales[f] = FP4 ? ws + r * (p.I / 32) : nullptr;
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int v = c * 16 + (lane & 15), i = least(v % half, n - 1);
        if constexpr (STAGED)
            a.at[c] = (v < half ? i : n + i) * column_bytes<FP4>(p.I);
        else
            a.col[c] = h + (int64_t)list[i].entry * p.I + (v < half ? 0 : p.lower);
    }
    int s0, s1;
    share(p.I, FP4 ? 4 : 1, wave, waves, s0, s1);
    if constexpr (STAGED) {
        stage_columns<FP4>(reinterpret_cast<char *>(red), h, 2 * p.lower, 2 * n, p.I, [&](int i) {
            return (int64_t)list[i < n ? i : i - n].entry * p.I + (i < n ? 0 : p.lower);
        });
        a.run(s0, s1, p.I);
        __syncthreads();        // `red` is the columns' memory
    } else {
        a.run(s0, s1, p.I);
    }
    a.put(red);
    __syncthreads();
    for (int i = tid; i < cols * least(n, half); i += blockDim.x) {
        const int c = i / cols, r = i % cols;
        if (r0 + r >= p.H)
            continue;
        const float v = joined(added<NT>(red, waves, r >> 4, c, r & 15), added<NT>(red, waves, r >> 4, half + c, r & 15));
        // read by a block on any XCD: not left in this one's L2
        __hip_atomic_store(part + (int64_t)list[c].entry * p.H + r0 + r, list[c].coef * v, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
}

template <bool FP4, int NT>
__device__ __forceinline__ void down_shared(const FewPlan &p, const uint16_t *h, const uint8_t *w, const uint8_t *ws,
                                            int e, int r0, const Token *list, int n, char *lds, float *part)
{
    constexpr int half = NT * 8;
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    Shared<FP4, NT> a;
    a.lds = lds;
    a.from = row_rsrc(h, (int)(2 * p.lower * 2));
    const int row = r0 + wave * 32;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int64_t r = (int64_t)e * p.H + least(row + f * 16 + (lane & 15), p.H - 1);
        a.w[f] = w + r * (FP4 ? p.I / 2 : p.I * 2);
        a.scales[f] = FP4 ? ws + r * (p.I / 32) : nullptr;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int c = (i * 4 + wave) * 4 + (lane >> 4), token = c % half;
        a.col[i] = token < n ? (uint32_t)(((int64_t)list[least(token, n - 1)].entry * p.I + (c < half ? 0 : p.lower)) * 2) +
                                   (((lane & 15) ^ (c & 15)) << 4)
                             : kNowhere;
    }
    a.run(p.I);
#pragma unroll
    for (int i = 0; i < (NT + 1) / 2; ++i) {
        const int c = i * 16 + (lane & 15);
        f32x4 sum[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (NT > 1)
                    sum[f][q] = joined(a.acc[f][i][q], a.acc[f][i + NT / 2][q]);
                else            // eight lanes on
                    sum[f][q] = joined(a.acc[f][0][q], dpp_f<0x128, 0xF>(0.0f, a.acc[f][0][q]));
            }
        }
        if (c >= least(n, half))
            continue;
        const Token t = list[c];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int at = row + f * 16 + (lane >> 4) * 4;
            const f32x4 v = t.coef * sum[f];
            uint64_t *to = reinterpret_cast<uint64_t *>(part + (int64_t)t.entry * p.H + at);
            if (at < p.H) {         // (H % 8 == 0)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    __hip_atomic_store(to + q, (uint64_t)__float_as_uint(v[2 * q + 1]) << 32 | __float_as_uint(v[2 * q]),
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
}

// The tokens' parts of the columns [r0, r0 + COLS), added up in the order of k: pairs of
// columns, U of them at a time and of each KC parts, all asked for together (a round is
// a miss to memory).
template <int U, int KC, int COLS>
__device__ __forceinline__ void add_parts(const FewPlan &p, const float *part, const uint64_t *firsts, int r0, uint16_t *out)
{
    const int all = p.T * (COLS / 2), step = blockDim.x;
    for (int i0 = threadIdx.x; i0 < all; i0 += U * step) {
        float a[U], b[U];
        uint64_t has[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = b[u] = 0.0f;
            const int i = i0 + u * step;
            has[u] = i < all && r0 + i % (COLS / 2) * 2 < p.H ? firsts[i / (COLS / 2)] : 0;
        }
        for (int k0 = 0; k0 < p.K; k0 += KC) {
            uint64_t v[U][KC];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    const int i = i0 + u * step;
                    const float *from = part + ((int64_t)(i / (COLS / 2)) * p.K + k0 + k) * p.H + r0 + i % (COLS / 2) * 2;
                    v[u][k] = 0;
                    if (k0 + k < p.K && has[u] >> (k0 + k) & 1)
                        v[u][k] = __hip_atomic_load(reinterpret_cast<const uint64_t *>(from), __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    a[u] += __uint_as_float((uint32_t)v[u][k]);
                    b[u] += __uint_as_float((uint32_t)(v[u][k] >> 32));
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step, c = r0 + i % (COLS / 2) * 2;
            if (i < all && c < p.H)
                *reinterpret_cast<uint32_t *>(out + (int64_t)(i / (COLS / 2)) * p.H + c) = pack_bf16_any(a[u], b[u]);
        }
    }
}

template <bool FP4, bool WIDE>
__global__ void __launch_bounds__(kMaxWaves *kWave, WIDE ? 2 : 4)
few_down_kernel(FewPlan p, const uint16_t *__restrict__ h, const int32_t *__restrict__ idx,
                const uint8_t *__restrict__ w, const uint8_t *__restrict__ ws, FewTables t, float *part,
                uint16_t *__restrict__ out)
{
    extern __shared__ __attribute__((aligned(16))) float red[];
    __shared__ Token list[kFewTokens];
    __shared__ bool last;
    constexpr int cols = WIDE ? 128 : 32;
    // tokens go 32 at a time, each lot to a block of its own; the first lots first.  (An
    // expert's blocks on one XCD, whose L2 would then have the columns once: 121 -> 129 us
    // with 128 tokens, 2 of 8 experts of unequal numbers.)
    const int tid = threadIdx.x, slice = blockIdx.x % p.slices, r0 = slice * cols;
    const int at = blockIdx.x / p.slices % p.most, lot = WIDE ? blockIdx.x / p.slices / p.most : 0;
    // (at < p.most: in the tables, if not of use)
    const int named = t.named[0], e = t.expert[at], n = t.count[at];
    const int total = t.named[1];
    // (before the numbers are here: what lies behind the n-th is of no use)
    for (int i = tid; i < p.T; i += blockDim.x)
        list[i] = Token{t.entry[at * p.T + i], t.coef[at * p.T + i]};
    if (named == 0 ? at + lot > 0 : at >= named || lot * 32 * WIDE >= n)
        return;
    if (named > 0) {
        __syncthreads();
        if constexpr (WIDE) {
            char *const lds = reinterpret_cast<char *>(red);
            const Token *mine = list + lot * 32;
            const int m = least(n - lot * 32, 32);
            if (m <= 8)
                down_shared<FP4, 1>(p, h, w, ws, e, r0, mine, m, lds, part);
            else if (m <= 16)
                down_shared<FP4, 2>(p, h, w, ws, e, r0, mine, m, lds, part);
            else
                down_shared<FP4, 4>(p, h, w, ws, e, r0, mine, m, lds, part);
        } else {
            if (n <= 8 && can_stage<FP4>(p, 2 * n, p.I, 2 * p.lower))
                down_group<FP4, 1, true>(p, h, w, ws, e, r0, list, n, red, part);
            else if (n <= 8)
                down_group<FP4, 1, false>(p, h, w, ws, e, r0, list, n, red, part);
            else
                for (int g = 0; g < n; g += 16)
                    down_group<FP4, 2, false>(p, h, w, ws, e, r0, list + g, n - g, red, part);
        }
    }
    // Every wave's parts have arrived where all XCDs see them before the block counts
    // itself, and the last block reads them there: the parts' accesses go past the
    // caches, so that no cache needs writing back or invalidating (which would
    // cost the other blocks what they have there of h).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // (it counts the tokens that it brings)
    if (tid == 0) {
        const unsigned brings = WIDE ? least(n - lot * 32, 32) : n;
        last = named == 0 || __hip_atomic_fetch_add(t.arrived + slice, brings, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT) + brings == (unsigned)total;
    }
    __syncthreads();
    if (!last)
        return;
    if (p.K <= 2)
        add_parts<WIDE ? 16 : 8, 2, cols>(p, part, t.firsts, r0, out);
    else
        add_parts<WIDE ? 4 : 2, 8, cols>(p, part, t.firsts, r0, out);
}

__global__ void few_zero_kernel(int32_t *p) { *p = 0; }

// The waves of a block, by the inner dimension: eight steps of 32 for each, or four of
// 128 (one token, H 7168, I 2048: 59.8 us, with six steps 61.2, with sixteen 63).
int waves_of(int D, bool fp4)
{
    const int steps = (D + (fp4 ? 127 : 31)) / (fp4 ? 128 : 32), per = fp4 ? 4 : 8;
    return steps >= 4 * per ? 4 : (steps >= 2 * per ? 2 : 1);
}

template <bool FP4, bool WIDE>
hipError_t launch_few_as(const FewPlan &p, const uint16_t *x, const int32_t *idx, const float *weights,
                         const uint8_t *up, const uint8_t *up_scales, const uint8_t *down, const uint8_t *down_scales,
                         const FewTables &t, uint16_t *h, float *part, uint16_t *out, int32_t *num_invalid,
                         hipStream_t s)
{
    const int wu = WIDE ? kMaxWaves : waves_of(p.H, FP4), wd = WIDE ? kMaxWaves : waves_of(p.I, FP4);
    // four buffers of 64 columns; or the waves' sums of 2 x 2 fragments, or the columns
    // and the entries
    auto lds = [&](int waves) {
        const int own = WIDE ? 4 * 4 * 4096 : waves * 4096 > p.stage_bytes ? waves * 4096 : p.stage_bytes;
        return own > p.T * p.K * 8 ? own : p.T * p.K * 8;
    };
    // beyond the 64 KB that a block has without asking
    const void *kernels[2] = {reinterpret_cast<const void *>(few_up_kernel<FP4, WIDE>),
                              reinterpret_cast<const void *>(few_down_kernel<FP4, WIDE>)};
    for (const void *k : kernels) {
        const hipError_t e = WIDE ? hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, lds(kMaxWaves))
                                  : hipSuccess;
        if (e != hipSuccess)
            return e;
    }
    const int lots_up = WIDE ? (p.T + 63) / 64 : 1, lots_down = WIDE ? (p.T + 31) / 32 : 1;
    few_up_kernel<FP4, WIDE><<<p.most * lots_up * p.slices_up, wu * kWave, lds(wu), s>>>(p, x, idx, weights, up, up_scales, t, h,
                                                                              num_invalid);
    few_down_kernel<FP4, WIDE><<<p.most * lots_down * p.slices, wd * kWave, lds(wd), s>>>(p, h, idx, down, down_scales, t, part, out);
    return hipGetLastError();
}

}  // namespace

FewPlan make_few_plan(int T, int K, int E, int H, int I, bool fp4)
{
    FewPlan p{};
    p.T = T;
    p.K = K;
    p.E = E;
    p.H = H;
    p.I = I;
    p.most = least(T * K, E);
    // Blocks of 128 weight rows, that share the tokens' columns (whose arrays a buffer has
    // to reach), or of 32.  Large ones need work for the card: tokens' entries times
    // blocks of an expert.  MXFP4 (us with 32 and with 128; T, K, E, H, I):
    //   4, 2, 8, 4096, 4096 (512 of them)      45   51    16, 4, 16, 4096, 1024 (1024)  52   38
    //   16, 4, 64, 2048, 512 (512)             36   31    8, 8, 64, 7168, 2048 (2048)  258  225
    //   16, 2, 8, 2048, 1024 (512)             23   27    80, 8, 64, 7168, 2048        757  433
    // bf16, whose rows' bytes keep the small ones busy, needs more tokens for each expert too:
    //   32, 8, 8, 1024, 512 (2048)             27   36    64, 8, 64, 4096, 1024        368  336
    //   48, 8, 64, 4096, 1024 (6144)          322  319    128, 8, 16, 2048, 1024       224  131
    //   16, 8, 64, 4096, 1024                 229  235    32, 2, 8, 4096, 4096         170  178
    const int64_t work = (int64_t)T * K * ((I + 63) / 64);
    p.wide = (int64_t)T * K * I < 1 << 29 && (fp4 ? work >= 1024 : work >= 4096 && T * K >= 8 * p.most);
    const int rows = p.wide ? 128 : 32;
    // what an expert's tokens take of LDS, on average; twice that at most
    const int mean = p.most > 0 ? (T * K + p.most - 1) / p.most : 0, wide = H > 2 * I ? H : 2 * I;
    const int64_t want = ((int64_t)2 * mean * (wide * 2 + 256 + 64) + 1023) / 1024 * 1024;
    p.stage_bytes = (int)(want < kStageBytes ? want : kStageBytes);
    p.slices = (H + rows - 1) / rows;
    p.slices_up = (I + rows / 2 - 1) / (rows / 2);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t entries = (size_t)T * K;
    p.lower = (int64_t)entries * I;
    p.off_arrived = take((size_t)((H + 31) / 32) * 4);      // (for either type of weights)
    p.off_named = take(8);
    p.off_expert = take((size_t)p.most * 4);
    p.off_count = take((size_t)p.most * 4);
    p.off_entry = take((size_t)p.most * T * 4);
    p.off_coef = take((size_t)p.most * T * 4);
    p.off_firsts = take((size_t)T * 8);
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
    t.firsts = reinterpret_cast<uint64_t *>(ws + p.off_firsts);
    uint16_t *h = reinterpret_cast<uint16_t *>(ws + p.off_h);
    float *part = reinterpret_cast<float *>(ws + p.off_part);
    const uint8_t *u = static_cast<const uint8_t *>(up), *d = static_cast<const uint8_t *>(down);
    if (up_scales && p.wide)
        return launch_few_as<true, true>(p, x, idx, weights, u, up_scales, d, down_scales, t, h, part, out, num_invalid, s);
    if (up_scales)
        return launch_few_as<true, false>(p, x, idx, weights, u, up_scales, d, down_scales, t, h, part, out, num_invalid, s);
    if (p.wide)
        return launch_few_as<false, true>(p, x, idx, weights, u, nullptr, d, nullptr, t, h, part, out, num_invalid, s);
    return launch_few_as<false, false>(p, x, idx, weights, u, nullptr, d, nullptr, t, h, part, out, num_invalid, s);
}

}  // namespace ep
