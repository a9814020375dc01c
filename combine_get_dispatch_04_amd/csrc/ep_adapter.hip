// ep_adapter.hip -- low-rank adapters beside a shared projection:
//   out_t = W x_t + sum_k c_tk B_e A_e x_t,   e = topk_idx[t,k],  c_tk = scale w_tk
// and its gradients, with v_tk = B_e^T d_t for the output's gradient d:
//   dx_t = W^T d_t + sum_k c_tk A_e^T v_tk      dA_e = sum c_tk v_tk x_t^T
//   dw_tk = scale <A_e x_t, v_tk>               dB_e = sum c_tk d_t (A_e x_t)^T
//
// Tokens go in tiles of BM.  A tile's list holds the adapters that its tokens
// name, ascending; its dense matrix U holds in row t, columns l*rp .. l*rp+r-1,
// c * (A_e x_t) for the l-th adapter of the list, 0 where the
// token does not name it (rp = r rounded up to 16, c summed over the entries
// that name it).  So the adapters' part of a tile is one more stretch of the
// inner dimension of the projection's own matrix product, over U and the
// list's B, and the gradients of A and B are products of U's and V's columns
// with the tile's rows of d and x.
//
// U and V are the operands of MFMAs, but not the caller's values: one rounding
// to bf16 (2^-8 of a value) would be as large as the result's own, and 1.4 times the
// gradients' error.  So they are two matrices of bf16 each, a value's
// nearest and what that left over, together within 2^-16 of it; a product with
// them is one with each.  At 4096 x 4096 x 4096, 2 of 8 adapters of rank 16,
// the second one costs 2 and 3 us of the two projections' 109 and 116, and 9 of
// the gradients' 34.
//
//   shrink     the lists, and every adapter's place in them; A_e x_t (or B_e^T d_t)
//              of every entry, MFMA over the list's rows, the inner dimension split
//              over blocks; fp32
//   gather     sums the splits, writes U (or V) and the fp32 sums; dw
//   project    the product with W, and U's stretch in front of it
//   grads      dA, dB
//
// Products of tokens and adapters that do not belong together meet zeros of
// U.  A zero does not stop an infinity or a NaN (of another token's row, or of
// another request's adapter): where a wave's sums over U are not all finite it
// takes them again with every such product left out.
#include "ep_common.h"
#include "ep_internal.h"

namespace ep {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int BK = 64;                 // inner elements per stage: two slices of 32, one MFMA each

// ---------------------------------------------------------------- LDS tiles
// A tile of rows with 64 consecutive inner elements: 8 pieces of 16 bytes per
// row, piece c of row r in slot c ^ (r & 7), so that the 16 rows a fragment
// reads at one c spread over the banks.
__device__ __forceinline__ int off_k(int row, int piece)
{
    return row * 128 + ((piece ^ (row & 7)) << 4);
}
// A tile of 64 inner rows with consecutive columns, read transposed: blocks
// of 64 columns, each 64 rows of 128 bytes, so that the loads fetch whole
// 128-byte lines of 8 rows at a time as above.  A row has 4 units of 16
// columns (32 bytes), unit u of row k in slot u ^ g(k).  A transposing read
// takes rows {0..3, 8..11, 16..19, 24..27} of one unit: the row's parity and
// g tell eight of them apart.
__device__ __forceinline__ int unit_swizzle(int k) { return ((k >> 1) & 1) | ((k >> 2) & 2); }
__device__ __forceinline__ int off_n(int k, int unit)
{
    return (unit >> 2) * (BK * 128) + k * 128 + (((unit & 3) ^ unit_swizzle(k)) << 5);
}
// A lane's operand of one 16 x 32 fragment: 8 consecutive inner elements from
// ks*32 + (lane >> 4)*8, of row (or column) lane & 15 of its 16.  The lane's
// own offset is worked out once (at_k, at_n); fragments, stages and halves are
// constants on top of it, as row0 is a multiple of 16 and g(k) the same for k,
// k + 4 and k + 32.
__device__ __forceinline__ int at_k(int ks, int lane)
{
    return off_k(lane & 15, ks * 4 + (lane >> 4));
}
__device__ __forceinline__ bf16x8 frag_k(const char *tile, int row0, int at)
{
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(tile + row0 * 128 + at));
}
__device__ __forceinline__ int at_n(int unit, int lane)
{
    return off_n((lane >> 4) * 8 + ((lane & 15) >> 2), unit) + (lane & 3) * 8;
}
__device__ __forceinline__ bf16x8 frag_n(const char *tile, int ks, int at)
{
    typedef __attribute__((address_space(3))) s16x4 *lds4_ptr;
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_ptr)(tile + at + ks * 32 * 128));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_ptr)(tile + at + (ks * 32 + 4) * 128));
    const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
}
// The operands of N neighbouring units at once, while loads into LDS are in
// flight: the compiler would wait for those before each transposing read of
// its own (it cannot tell their buffers apart), so the reads and their wait are
// one block of assembly.  `at` is unit 0's address; unit j's differs in bits 5
// and 6, the other half of a fragment lies 4 rows (512 bytes) on, slice 1 32
// rows (4096 bytes).
template <int KS>
__device__ __forceinline__ void frags_n(const char *tile, int at, bf16x8 (&b)[4])
{
    typedef __attribute__((address_space(3))) const char *lds_char;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_char)tile;
    const uint32_t p0 = base + at, p1 = base + (at ^ 32), p2 = base + (at ^ 64), p3 = base + (at ^ 96);
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    u2 r0, r1, r2, r3, r4, r5, r6, r7;
    asm volatile("ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
                 "ds_read_b64_tr_b16 %2, %9 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
                 "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
                 "ds_read_b64_tr_b16 %6, %11 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(r0), "=&v"(r1), "=&v"(r2), "=&v"(r3), "=&v"(r4), "=&v"(r5), "=&v"(r6), "=&v"(r7)
                 : "v"(p0), "v"(p1), "v"(p2), "v"(p3), "n"(KS * 4096), "n"(KS * 4096 + 512)
                 : "memory");
    b[0] = __builtin_bit_cast(bf16x8, u32x4{r0[0], r0[1], r1[0], r1[1]});
    b[1] = __builtin_bit_cast(bf16x8, u32x4{r2[0], r2[1], r3[0], r3[1]});
    b[2] = __builtin_bit_cast(bf16x8, u32x4{r4[0], r4[1], r5[0], r5[1]});
    b[3] = __builtin_bit_cast(bf16x8, u32x4{r6[0], r6[1], r7[0], r7[1]});
}
template <int KS>
__device__ __forceinline__ void frags_n(const char *tile, int at, bf16x8 (&b)[2])
{
    typedef __attribute__((address_space(3))) const char *lds_char;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_char)tile;
    const uint32_t p0 = base + at, p1 = base + (at ^ 32);
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    u2 r0, r1, r2, r3;
    asm volatile("ds_read_b64_tr_b16 %0, %4 offset:%6\n\t"
                 "ds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
                 "ds_read_b64_tr_b16 %2, %5 offset:%6\n\t"
                 "ds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(r0), "=&v"(r1), "=&v"(r2), "=&v"(r3)
                 : "v"(p0), "v"(p1), "n"(KS * 4096), "n"(KS * 4096 + 512)
                 : "memory");
    b[0] = __builtin_bit_cast(bf16x8, u32x4{r0[0], r0[1], r1[0], r1[1]});
    b[1] = __builtin_bit_cast(bf16x8, u32x4{r2[0], r2[1], r3[0], r3[1]});
}
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------- a block's product
// BM tokens x BN columns, WM x WN waves.  acc[i][j]: token i*16 + (lane & 15)
// of the wave's rows, columns j*16 + (lane >> 4)*4 ..+3 of its columns.  The
// tokens' operand always has consecutive inner elements; the other one has
// them too (NN = false: rows of W, A_e) or lies across (NN = true: W read as
// its transpose).
//
// A stage goes from memory straight to LDS, into one of NS buffers, up to NS
// stages ahead of the MFMAs.  The wave's 64 pieces of 16 bytes land one after
// the other, so the swizzle is in the addresses: a lane fetches the piece that
// belongs into its slot.  The MFMAs go in TI groups of TJ, one row of
// fragments each; after a group the row's fragment of the next slice is read
// into the same registers, and a few of the next stage's loads are started:
// each keeps its own unit busy, and a wave that handed over all its loads at
// once would keep the matrix pipe waiting for the memory pipe to take them.
// One barrier per stage, some groups into its second slice, when every wave
// holds the rest of the stage in registers: its buffer is free.
typedef __attribute__((address_space(1))) const void *global_ptr;
typedef __attribute__((address_space(3))) void *lds_ptr;

template <int N>
__device__ __forceinline__ void wait_and_meet()     // at most N loads in flight, no LDS access
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int BM_, int BN_, int WM_, int WN_, int NS_, bool NN>
struct Product {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
    static constexpr int threads = WM * WN * kWave;
    static constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
    static constexpr int bytes_a = BM * BK * 2, bytes_b = BN * BK * 2;
    static constexpr int bytes = bytes_a + bytes_b, lds_bytes = NS * bytes;
    static constexpr int PA = BM * 8 / threads, PB = BN * 8 / threads;
    static_assert(PA * threads == BM * 8 && PB * threads == BN * 8, "whole pieces per thread");

    f32x4 acc[TI][TJ];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // What piece q of a buffer holds: row and first inner element (tokens, and
    // columns if NN = false) ...
    static __device__ __forceinline__ int row_of(int q) { return q >> 3; }
    static __device__ __forceinline__ int k_of(int q) { return ((q & 7) ^ (row_of(q) & 7)) * 8; }
    // ... or inner row and first column (NN = true).
    static __device__ __forceinline__ int kn_of(int q) { return q / 8 % BK; }
    static __device__ __forceinline__ int n_of(int q)
    {
        return q / (BK * 8) * 64 + ((q % 8 >> 1) ^ unit_swizzle(kn_of(q))) * 16 + (q & 1) * 8;
    }
    // Starts the load of the thread's piece number i of a stage into `buf`
    // (the tokens' operand first; `buf` moved on to the wave's pieces, see run):
    // pa(i), pb(i) are the pieces' addresses.
    static constexpr int pieces = PA + PB;
    template <typename FA, typename FB>
    static __device__ __forceinline__ void fetch(char *buf, int i, FA pa, FB pb)
    {
        if (i < PA)
            __builtin_amdgcn_global_load_lds((global_ptr)pa(i), (lds_ptr)(buf + i * threads * 16), 16, 0, 0);
        else
            __builtin_amdgcn_global_load_lds((global_ptr)pb(i - PA),
                                             (lds_ptr)(buf + bytes_a + (i - PA) * threads * 16), 16, 0, 0);
    }
    // The same through registers, for a stage that ends beyond the inner
    // dimension: va(p), vb(p) give the pieces, zeros where there is nothing.
    template <typename FA, typename FB>
    static __device__ __forceinline__ void fill(char *buf, FA va, FB vb)
    {
#pragma unroll 1
        for (int p = 0; p < PA; ++p)
            *reinterpret_cast<u32x4 *>(buf + (p * threads + threadIdx.x) * 16) = va(p);
#pragma unroll 1
        for (int p = 0; p < PB; ++p)
            *reinterpret_cast<u32x4 *>(buf + bytes_a + (p * threads + threadIdx.x) * 16) = vb(p);
    }
    // A lane's offsets of the wave's first fragments in a buffer.  Slice 1 of
    // consecutive inner elements differs from slice 0 in bit 6.
    struct Place {
        int a, b;
    };
    static __device__ __forceinline__ Place place()
    {
        const int lane = threadIdx.x & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int wm = wave / WN, wn = wave % WN;
        return {wm * (BM / WM) * 128 + at_k(0, lane),
                bytes_a + (NN ? at_n(wn * (BN / WN / 16), lane) : wn * (BN / WN) * 128 + at_k(0, lane))};
    }
    template <int KS>
    static __device__ __forceinline__ void read_b(bf16x8 (&b)[TJ], const char *buf, const Place &w)
    {
        if constexpr (NN) {
            frags_n<KS>(buf, w.b, b);
        } else {
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                b[j] = frag_k(buf, j * 16, w.b ^ (KS * 64));
        }
    }
    template <int KS>
    static __device__ __forceinline__ bf16x8 read_a(int i, const char *buf, const Place &w)
    {
        return frag_k(buf, i * 16, w.a ^ (KS * 64));
    }
    __device__ __forceinline__ void group(int i, const bf16x8 (&a)[TI], const bf16x8 (&b)[TJ])
    {
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            acc[i][j] = mfma(b[j], a[i], acc[i][j]);
    }
    // Groups [FROM, TI) of a slice; after them, spread out, the reads of the
    // next slice (KS of `from`; a[0 .. FROM) too) and the loads of a stage into
    // `to`.
    template <int FROM, int KS, bool FETCH, typename FF>
    __device__ __forceinline__ void groups(bf16x8 (&a)[TI], const bf16x8 (&b)[TJ], bf16x8 (&b_next)[TJ],
                                           const char *from, const Place &w, char *to, FF &fetch_piece)
    {
        constexpr int n = TI - FROM, RF = (pieces + n - 1) / n;
#pragma unroll
        for (int g = 0; g < n; ++g) {
            group(FROM + g, a, b);
            // not before these MFMAs, which would wait for the reads as well
            __builtin_amdgcn_sched_barrier(0);
            if (g == 0)
                read_b<KS>(b_next, from, w);
#pragma unroll
            for (int i = g == 0 ? 0 : FROM + g; i <= FROM + g; ++i)
                a[i] = read_a<KS>(i, from, w);
            if constexpr (FETCH) {
#pragma unroll
                for (int f = g * RF; f < (g + 1) * RF && f < pieces; ++f)
                    fetch_piece(to, f);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // Stages [0, n): fetch_piece(buf, i) starts the load of piece i of the next
    // stage, advance() goes on to the one after it.  Ends with every buffer free.
    template <typename FF, typename FN>
    __device__ __forceinline__ void run(char *lds, int n, FF fetch_piece, FN advance)
    {
        constexpr int LAG = TI > 2 ? 2 : 1;
        if (n <= 0)
            return;
        const Place w = place();
        // where the wave's pieces go, in scalar registers for the loads into LDS
        char *const mine = lds + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * (kWave * 16);
        for (int s = 0; s < NS && s < n; ++s) {
#pragma unroll
            for (int i = 0; i < pieces; ++i)
                fetch_piece(mine + s * bytes, i);
            advance();
        }
        if (n >= NS)
            wait_and_meet<(NS - 1) * pieces>();
        else
            wait_and_meet<0>();
        bf16x8 a[TI], b0[TJ], b1[TJ];
        read_b<0>(b0, lds, w);
#pragma unroll
        for (int i = 0; i < TI; ++i)
            a[i] = read_a<0>(i, lds, w);
        int cur = 0, s = 0;
        for (; s + NS < n; ++s) {
            const int nxt = cur + 1 == NS ? 0 : cur + 1;
            char *buf = lds + cur * bytes;
            groups<0, 1, false>(a, b0, b1, buf, w, buf, fetch_piece);
#pragma unroll
            for (int i = 0; i < LAG; ++i)
                group(i, a, b1);
            wait_and_meet<(NS - 2) * pieces>();
            groups<LAG, 0, true>(a, b1, b0, lds + nxt * bytes, w, mine + cur * bytes, fetch_piece);
            advance();
            cur = nxt;
        }
#pragma unroll 1
        for (; s < n; ++s) {
            const int nxt = cur + 1 == NS ? 0 : cur + 1;
            char *buf = lds + cur * bytes;
            groups<0, 1, false>(a, b0, b1, buf, w, buf, fetch_piece);
#pragma unroll
            for (int i = 0; i < LAG; ++i)
                group(i, a, b1);
            wait_and_meet<0>();
            // behind the last stage: a buffer that is not used any more
            groups<LAG, 0, false>(a, b1, b0, lds + nxt * bytes, w, buf, fetch_piece);
            cur = nxt;
        }
        wait_and_meet<0>();
    }
    // One stage through registers (fill).
    template <typename FA, typename FB>
    __device__ __forceinline__ void run_filled(char *lds, FA va, FB vb)
    {
        const Place w = place();
        fill(lds, va, vb);
        __syncthreads();
        bf16x8 a[TI], b[TJ];
        read_b<0>(b, lds, w);
#pragma unroll
        for (int i = 0; i < TI; ++i)
            a[i] = read_a<0>(i, lds, w);
#pragma unroll
        for (int i = 0; i < TI; ++i)
            group(i, a, b);
        read_b<1>(b, lds, w);
#pragma unroll
        for (int i = 0; i < TI; ++i)
            a[i] = read_a<1>(i, lds, w);
#pragma unroll
        for (int i = 0; i < TI; ++i)
            group(i, a, b);
        __syncthreads();
    }
    __device__ __forceinline__ bool finite() const
    {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    s = fmaf(acc[i][j][q], 0.0f, s);
        return s == 0.0f;       // an infinity or a NaN anywhere makes it NaN
    }
};

__host__ __device__ __forceinline__ int least(int a, int b) { return a < b ? a : b; }

// Blocks are dealt to the 8 XCDs in turn; this gives each XCD a run of
// consecutive tiles, so that its L2 sees the operands they share.
__device__ __forceinline__ int xcd_order(int b, int n)
{
    const int each = n / 8, rest = n % 8, x = b % 8;
    return x * each + least(x, rest) + b / 8;
}

// ---------------------------------------------------------------- tiles
struct Tiles {
    int T, K, E, r, rp, BM, Lmax, LW;
    const int32_t *idx;         // [T, K]
    int32_t *cnt;               // [ntile] adapters in the list
    int32_t *list;              // [ntile, Lmax]
    int32_t *place;             // [ntile, E] place in the list, or -1
    int32_t *bad;               // [ntile] invalid entries
    int64_t low;                // a dense matrix's lower part, so many elements behind the upper one
};

__device__ __forceinline__ u32x4 zero4() { return u32x4{0u, 0u, 0u, 0u}; }

// A tile's list, built by a block of at least 128 threads into shared memory
// (`list`, with bits and firsts of 128 words each); with `write` also to memory,
// with the places and the invalid entries' count.  Every block of a tile makes its
// own: that is cheaper than a launch before it.
constexpr int kListWords = 4096 / 32;       // most adapters
__device__ int build_list(const Tiles &m, int tile, int32_t *list, uint32_t *bits, int32_t *firsts,
                          bool write)
{
    const int tid = threadIdx.x, bd = blockDim.x;
    const int words = (m.E + 31) / 32;
    __shared__ int n_bad;
    if (tid < kListWords)
        bits[tid] = 0u;
    if (tid == 0)
        n_bad = 0;
    __syncthreads();
    const int t0 = tile * m.BM, t1 = m.T - t0 < m.BM ? m.T : t0 + m.BM;
    int bad = 0;
    for (int64_t i = (int64_t)t0 * m.K + tid; i < (int64_t)t1 * m.K; i += bd) {
        const int e = m.idx[i];
        if ((unsigned)e < (unsigned)m.E)
            atomicOr(&bits[e >> 5], 1u << (e & 31));
        else
            bad += e != -1;
    }
    if (bad)
        atomicAdd(&n_bad, bad);
    __syncthreads();
    if (tid < kWave) {                  // two words a lane
        const int c0 = __popc(bits[2 * tid]), c1 = __popc(bits[2 * tid + 1]);
        const int upto = wave_inclusive_scan(c0 + c1, tid);
        firsts[2 * tid] = upto - c0 - c1;
        firsts[2 * tid + 1] = upto - c1;
        if (tid == kWave - 1)
            firsts[kListWords] = upto;
    }
    __syncthreads();
    if (tid < words) {
        int at = firsts[tid];
        for (uint32_t b = bits[tid]; b; b &= b - 1u)
            list[at++] = tid * 32 + __ffs(b) - 1;
    }
    __syncthreads();
    const int n = firsts[kListWords];
    if (write) {
        for (int i = tid; i < n; i += bd)
            m.list[(int64_t)tile * m.Lmax + i] = list[i];
        for (int e = tid; e < m.E; e += bd) {
            const uint32_t b = bits[e >> 5], one = 1u << (e & 31);
            m.place[(int64_t)tile * m.E + e] = b & one ? firsts[e >> 5] + __popc(b & (one - 1u)) : -1;
        }
        if (tid == 0) {
            m.cnt[tile] = n;
            m.bad[tile] = n_bad;
        }
    }
    return n;
}
// The list that an earlier launch made, into shared memory: the addresses of
// loads into LDS go by it, and a wait for a list entry from memory would be one
// for those loads too.
__device__ __forceinline__ int load_list(const Tiles &m, int tile, int32_t *list)
{
    const int n = m.cnt[tile];
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        list[i] = m.list[(int64_t)tile * m.Lmax + i];
    __syncthreads();
    return n;
}

__global__ void adapter_zero_kernel(int32_t *p) { *p = 0; }

// How a tile's `slots` blocks share a list of `cols` columns: chunks of 128
// columns, or of 64 for a short list (the tokens' rows are read once per chunk);
// blocks beyond the chunks split the inner dimension, into `deep` parts at most.
__device__ __forceinline__ int shrink_width(int cols) { return cols > 64 ? 128 : 64; }
__device__ __forceinline__ int shrink_chunks(int cols)
{
    return (cols + shrink_width(cols) - 1) / shrink_width(cols);
}
__device__ __forceinline__ int shrink_splits(int cols, int slots, int deep)
{
    const int chunks = shrink_chunks(cols);
    return chunks >= slots || chunks == 0 ? 1 : least(slots / chunks, deep);
}
// Parts of about 4 stages.
__host__ __device__ __forceinline__ int shrink_depth(int D) { return D < 8 * BK ? 1 : D / (4 * BK); }

// ---------------------------------------------------------------- shrink
// part[split][t*K + k][r] = sum over the split's inner elements of src[t][.]
// times the entry's adapter: A [E, r, D] (NN = false), or B [E, D, r] (NN =
// true).  Products of a token and an adapter it does not name are dropped.
// One chunk of the list's columns, from column n0, for tokens t0 ..
template <typename P, bool NN>
__device__ __forceinline__ void shrink_chunk(const Tiles &m, const uint16_t *src, const uint16_t *ad, int D,
                                             const int32_t *list, int cols, int t0, int n0, int s0, int s1,
                                             int split, float *part, char *lds)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int whole = least(s1, D / BK) - s0;       // without the stage that ends beyond D
    P p;
    p.zero();
    // rows behind the last token and columns behind the list's last repeat
    // a row and a column that exist: their products are not stored
    const uint16_t *pa[P::PA], *pb[P::PB];
#pragma unroll
    for (int i = 0; i < P::PA; ++i) {
        const int q = i * P::threads + tid;
        pa[i] = src + (int64_t)least(t0 + P::row_of(q), m.T - 1) * D + (s0 * BK + P::k_of(q));
    }
#pragma unroll
    for (int i = 0; i < P::PB; ++i) {
        const int q = i * P::threads + tid;
        const int n = n0 + (NN ? P::n_of(q) : P::row_of(q));
        const int l = n < cols ? n / m.rp : 0, j = n < cols && n % m.rp < m.r ? n % m.rp : 0;
        const int64_t e = list[l];
        pb[i] = NN ? ad + (e * D + s0 * BK + P::kn_of(q)) * m.r + j
                   : ad + (e * m.r + j) * D + (s0 * BK + P::k_of(q));
    }
    p.run(lds, whole, [&](char *buf, int i) {
        P::fetch(buf, i, [&](int i) { return pa[i]; }, [&](int i) { return pb[i]; });
    }, [&] {
#pragma unroll
        for (int i = 0; i < P::PA; ++i)
            pa[i] += BK;
#pragma unroll
        for (int i = 0; i < P::PB; ++i)
            pb[i] += NN ? BK * m.r : BK;
    });
    if (whole < s1 - s0) {
        const int k0 = (s0 + whole) * BK, left = D - k0;
        p.run_filled(
            lds,
            [&](int i) {
                const int q = i * P::threads + tid, k = P::k_of(q);
                return k < left ? ld16(src + (int64_t)least(t0 + P::row_of(q), m.T - 1) * D + k0 + k)
                                : zero4();
            },
            [&](int i) {
                const int q = i * P::threads + tid;
                const int n = n0 + (NN ? P::n_of(q) : P::row_of(q));
                const int k = NN ? P::kn_of(q) : P::k_of(q);
                if (k >= left || n >= cols || n % m.rp >= m.r)
                    return zero4();
                const int64_t e = list[n / m.rp];
                return NN ? ld16(ad + (e * D + k0 + k) * m.r + n % m.rp)
                          : ld16(ad + (e * m.r + n % m.rp) * D + k0 + k);
            });
    }
    // a lane's columns: four of one adapter per fragment, -1 where there is none
    int e_of[P::TJ], j_of[P::TJ];
#pragma unroll
    for (int j = 0; j < P::TJ; ++j) {
        const int n = n0 + wave % P::WN * (P::BN / P::WN) + j * 16 + (lane >> 4) * 4;
        j_of[j] = n % m.rp;
        e_of[j] = n < cols && j_of[j] < m.r ? list[n / m.rp] : -1;
    }
    // the entries are read once each, and before the stores, which for all the
    // compiler knows might be to them (read again for every fragment, the kernel
    // takes 1.35 times as long at 4096 x 4096, K = 2)
    const int ta = t0 + wave / P::WN * (P::BM / P::WM) + (lane & 15);
    for (int k = 0; k < m.K; ++k) {
        int named[P::TI];
#pragma unroll
        for (int i = 0; i < P::TI; ++i)
            named[i] = ta + i * 16 < m.T ? m.idx[(int64_t)(ta + i * 16) * m.K + k] : -2;
#pragma unroll
        for (int i = 0; i < P::TI; ++i) {
            float *o = part + (((int64_t)split * m.T + ta + i * 16) * m.K + k) * m.r;
#pragma unroll
            for (int j = 0; j < P::TJ; ++j)
                if (e_of[j] >= 0 && e_of[j] == named[i])
                    *reinterpret_cast<f32x4 *>(o + j_of[j]) = p.acc[i][j];
        }
    }
}

// A block takes RB tokens of a tile.
template <int RB, bool NN>
struct Shrink {
    typedef Product<RB, 64, RB / 32, 1, 3, NN> Narrow;
    typedef Product<RB, 128, RB / 64, 2, 2, NN> Wide;
    static constexpr int lds_bytes = Narrow::lds_bytes > Wide::lds_bytes ? Narrow::lds_bytes : Wide::lds_bytes;
};
template <int RB, bool NN>
__global__ void __launch_bounds__(RB * 2, 2)
adapter_shrink_kernel(Tiles m, const uint16_t *__restrict__ src, const uint16_t *__restrict__ ad,
                      int D, int slots, float *__restrict__ part)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    typedef Shrink<RB, NN> S;
    static_assert(S::Narrow::threads == RB * 2 && S::Wide::threads == RB * 2, "one block shape");
    const int block = blockIdx.x / slots, slot = blockIdx.x % slots;
    const int tile = block / (m.BM / RB), t0 = block * RB;
    if (t0 >= m.T)
        return;
    int32_t *list = reinterpret_cast<int32_t *>(lds + S::lds_bytes);
    __shared__ uint32_t bits[kListWords];
    __shared__ int32_t firsts[kListWords + 1];
    const int cols = m.rp * (NN ? load_list(m, tile, list)
                                : build_list(m, tile, list, bits, firsts, slot == 0 && t0 == tile * m.BM));
    const int chunks = shrink_chunks(cols), splits = shrink_splits(cols, slots, shrink_depth(D));
    const int split = chunks >= slots ? 0 : (chunks > 0 ? slot / chunks : 0);
    if (split >= splits)
        return;
    const int step = chunks >= slots ? slots : chunks;
    const int steps = (D + BK - 1) / BK;
    const int s0 = (int)((int64_t)steps * split / splits);
    const int s1 = (int)((int64_t)steps * (split + 1) / splits);
    for (int chunk = chunks >= slots ? slot : (chunks > 0 ? slot % chunks : 0); chunk < chunks;
         chunk += step) {
        if (cols > 64)
            shrink_chunk<typename S::Wide, NN>(m, src, ad, D, list, cols, t0, chunk * 128, s0, s1, split, part, lds);
        else
            shrink_chunk<typename S::Narrow, NN>(m, src, ad, D, list, cols, t0, 0, s0, s1, split, part, lds);
        __syncthreads();        // the buffers are free for the next chunk
    }
}

// ---------------------------------------------------------------- gather
// Sums the splits: sums[t*K + k][r] in fp32, and both parts of the tile's dense
// matrix, zeros up to the next 64 columns.  With `u` given, dw[t,k] = scale <u, sums>.
// A block takes 32 rows of a tile.  Latency: three loads one after the other (5 to 6 us).
constexpr int kGatherRows = 32;
// What two values lost in their bf16 forms `v`; nothing if those are not finite.
__device__ __forceinline__ uint32_t lower_part(float a, float b, uint32_t v)
{
    const float da = a - bf16_lo(v), db = b - bf16_hi(v);
    return pack_bf16_any(fabsf(da) < __builtin_huge_valf() ? da : 0.0f,
                         fabsf(db) < __builtin_huge_valf() ? db : 0.0f);
}
constexpr int kDensePad = BK;          // the project kernel takes whole stages of U
__global__ void __launch_bounds__(256)
adapter_gather_kernel(Tiles m, const float *__restrict__ w, float scale, int slots, int deep,
                      const float *__restrict__ part, float *__restrict__ sums,
                      uint16_t *__restrict__ dense, const float *__restrict__ u,
                      float *__restrict__ dw, int ntile, int32_t *__restrict__ num_invalid)
{
    const int per = m.BM / kGatherRows;
    const int tile = blockIdx.x / per, row0 = (blockIdx.x % per) * kGatherRows;
    const int tid = threadIdx.x;
    const int cols = m.cnt[tile] * m.rp;
    const int pieces = (cols + kDensePad - 1) / kDensePad * (kDensePad / 8);
    const int splits = shrink_splits(cols, slots, deep);
    const int64_t stride = (int64_t)m.T * m.K * m.r;
    // zeros, then the entries' own columns
    for (int i = tid; i < kGatherRows * pieces; i += 256) {
        uint16_t *o = dense + ((int64_t)tile * m.BM + row0 + i / pieces) * m.LW + i % pieces * 8;
        st16(o, zero4());
        st16(o + m.low, zero4());
    }
    __syncthreads();
    const int per_row = m.K * (m.r / 8);
    for (int i = tid; i < kGatherRows * per_row; i += 256) {
        const int t = tile * m.BM + row0 + i / per_row;
        if (t >= m.T)
            break;
        const int k = i % per_row / (m.r / 8), j = i % (m.r / 8) * 8;
        const int64_t t0 = (int64_t)t * m.K, tk = t0 + k;
        const int e = m.idx[tk];
        if ((unsigned)e >= (unsigned)m.E)
            continue;
        const float *p = part + tk * m.r + j;
        f32x4 lo = {0.0f, 0.0f, 0.0f, 0.0f}, hi = lo;
#pragma unroll 8
        for (int q = 0; q < splits; ++q) {
            lo += *reinterpret_cast<const f32x4 *>(p + q * stride);
            hi += *reinterpret_cast<const f32x4 *>(p + q * stride + 4);
        }
        const int l = m.place[(int64_t)tile * m.E + e];
        // the coefficients of all entries that name e; the first one writes
        float coef = 0.0f;
        bool first = true;
        for (int o = 0; o < m.K; ++o)
            if (m.idx[t0 + o] == e) {
                coef += w ? w[t0 + o] : 1.0f;
                first = first && o >= k;
            }
        float *o = sums + tk * m.r + j;
        *reinterpret_cast<f32x4 *>(o) = lo;
        *reinterpret_cast<f32x4 *>(o + 4) = hi;
        if (!first)
            continue;
        lo *= scale * coef;
        hi *= scale * coef;
        const u32x4 v = {pack_bf16_any(lo[0], lo[1]), pack_bf16_any(lo[2], lo[3]),
                         pack_bf16_any(hi[0], hi[1]), pack_bf16_any(hi[2], hi[3])};
        uint16_t *to = dense + (int64_t)t * m.LW + l * m.rp + j;
        st16(to, v);
        st16(to + m.low, u32x4{lower_part(lo[0], lo[1], v[0]), lower_part(lo[2], lo[3], v[1]),
                               lower_part(hi[0], hi[1], v[2]), lower_part(hi[2], hi[3], v[3])});
    }
    if (u && dw) {
        __syncthreads();        // the block's own sums are read back
        for (int i = tid; i < kGatherRows * m.K; i += 256) {
            const int t = tile * m.BM + row0 + i / m.K;
            if (t >= m.T)
                break;
            const int64_t tk = (int64_t)t * m.K + i % m.K;
            f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
            if ((unsigned)m.idx[tk] < (unsigned)m.E) {
#pragma unroll 4
                for (int j = 0; j < m.r; j += 4) {
                    const f32x4 a = *reinterpret_cast<const f32x4 *>(u + tk * m.r + j);
                    const f32x4 b = *reinterpret_cast<const f32x4 *>(sums + tk * m.r + j);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        d[q] = fmaf(a[q], b[q], d[q]);
                }
            }
            dw[tk] = scale * ((d[0] + d[1]) + (d[2] + d[3]));
        }
    }
    if (num_invalid && blockIdx.x == 0 && tid < kWave) {
        int n = 0;
        for (int i = tid; i < ntile; i += kWave)
            n += m.bad[i];
        n = wave_sum(n);
        if (tid == 0)
            num_invalid[0] = n;
    }
}

// ---------------------------------------------------------------- project
// out[t][n] = sum_l dense[t][l] adapter_l[.][n] + sum_k src[t][k] W: W [N, D]
// and B [E, N, r] for the forward (NN = false), W [D, N] and A [E, r, N] for
// the gradient of x (NN = true).
// Measured in a steady stream of calls: 4096 x 4096 x 4096 with eight adapters of
// rank 16 in every tile 109 us (1.26 PFLOP/s) and 116 us (NN), 4001 x 7168 x 7168
// 321 us, 346 where the gradient's product runs in turn with it (1.28 and 1.19
// PFLOP/s); without adapters no less.  Bound by the matrix pipes, busy 58 % of the
// time (52 % NN), with the waves at a wait for 25 to 33 % of theirs and at a pipe
// that is taken for 50 % (with half of the loads left out 102 us of 105, with a
// quarter of the MFMAs 79).

// The adapters' part of 16 tokens (lane & 15: token t with its row u of U) by
// columns c .. c+15, one adapter at a time, each for the tokens that name it
// only: where the sum over U is not finite.  A sum over the upper part that is not
// finite stands alone: the lower part may have other signs, and infinities of
// both would be a NaN.
template <bool NN>
__device__ __forceinline__ f32x4 adapters_apart(const Tiles &m, const int32_t *list, int n_list,
                                                const uint16_t *u, int t, const uint16_t *ad, int N,
                                                int c, int lane)
{
    const int n = c + (lane & 15);
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int l = 0; l < n_list; ++l) {
        const int64_t e = list[l];
        bool named = false;
        for (int k = 0; t < m.T && k < m.K; ++k)
            named = named || m.idx[(int64_t)t * m.K + k] == (int)e;
        f32x4 one = {0.0f, 0.0f, 0.0f, 0.0f}, rest = one;
#pragma unroll 1
        for (int k0 = 0; k0 < m.rp; k0 += 32) {
            const int k = k0 + (lane >> 4) * 8;
            u32x4 fu = zero4(), fl = zero4(), fa = zero4();
            if (k < m.r) {
                fu = ld16(u + l * m.rp + k);
                fl = ld16(u + m.low + l * m.rp + k);
                if (n < N) {
                    if constexpr (NN) {
                        const uint16_t *a = ad + (e * m.r + k) * N + n;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            fa[q] = a[(2 * q) * (int64_t)N] | ((uint32_t)a[(2 * q + 1) * (int64_t)N] << 16);
                    } else {
                        fa = ld16(ad + (e * N + n) * m.r + k);
                    }
                }
            }
            one = mfma(__builtin_bit_cast(bf16x8, fa), __builtin_bit_cast(bf16x8, fu), one);
            rest = mfma(__builtin_bit_cast(bf16x8, fa), __builtin_bit_cast(bf16x8, fl), rest);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (named)
                sum[q] += fabsf(one[q]) < __builtin_huge_valf() ? one[q] + rest[q] : one[q];
    }
    return sum;
}

template <typename P, bool NN>
__global__ void __launch_bounds__(P::threads, 2)     // two waves per SIMD at least
adapter_project_kernel(Tiles m, const uint16_t *__restrict__ src, int D,
                       const uint16_t *__restrict__ weight, int N, const uint16_t *__restrict__ ad,
                       const uint16_t *__restrict__ dense, int ntile, uint16_t *__restrict__ out)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int BM = P::BM, BN = P::BN, WM = P::WM, WN = P::WN;
    // tiles in groups of 8 token tiles by all columns, column by column
    const int nb = (N + BN - 1) / BN;
    const int id = xcd_order(blockIdx.x, ntile * nb);
    const int group = id / (8 * nb), first = group * 8;
    const int rows = least(8, ntile - first);
    const int tile = first + (id - group * 8 * nb) % rows, n0 = (id - group * 8 * nb) / rows * BN;
    const int t0 = tile * BM;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int wm = wave / WN, wn = wave % WN;
    int32_t *list = reinterpret_cast<int32_t *>(lds + P::lds_bytes);
    const int cols = load_list(m, tile, list) * m.rp;
    const uint16_t *du = dense + (int64_t)t0 * m.LW;
    P p;
    p.zero();
    bool apart = false;
    if (cols > 0) {
        // columns behind the list's last meet zeros of U.  A piece's place in the
        // list and in its adapter goes on by a stage without dividing again.
        int l[P::PB], j[P::PB];
#pragma unroll
        for (int i = 0; i < P::PB; ++i) {
            const int q = i * P::threads + tid, k = NN ? P::kn_of(q) : P::k_of(q);
            l[i] = k / m.rp;
            j[i] = k % m.rp;
        }
        const int whole = BK / m.rp, rest = BK % m.rp, n_list = cols / m.rp;
        int k0 = 0;
        int64_t part = 0;       // every stage with the upper part, then with the lower one
        p.run(lds, (cols + BK - 1) / BK * 2, [&](char *buf, int i) {
            P::fetch(
                buf, i,
                [&](int i) {
                    const int q = i * P::threads + tid;
                    return du + part + (int64_t)P::row_of(q) * m.LW + k0 + P::k_of(q);
                },
                [&](int i) {
                    const int q = i * P::threads + tid;
                    const int64_t e = list[least(l[i], n_list - 1)];
                    const int c = j[i] < m.r ? j[i] : 0;
                    return NN ? ad + (e * m.r + c) * N + least(n0 + P::n_of(q), N - 8)
                              : ad + (e * N + least(n0 + P::row_of(q), N - 1)) * m.r + c;
                });
        }, [&] {
            part = part ? 0 : m.low;
            if (part)
                return;
            k0 += BK;
#pragma unroll
            for (int i = 0; i < P::PB; ++i) {
                const bool over = j[i] + rest >= m.rp;
                l[i] += whole + over;
                j[i] += over ? rest - m.rp : rest;
            }
        });
        apart = __any(!p.finite());
        if (apart)
            p.zero();
    }
    {
        // the block's first row of each operand, which moves along, and the
        // pieces' byte offsets from there, which stay (32 bits: H and O are at
        // most 2^20); rows and columns behind the last repeat one that exists
        const char *ba = reinterpret_cast<const char *>(src + (int64_t)t0 * D);
        const char *bb = reinterpret_cast<const char *>(NN ? weight + n0 : weight + (int64_t)n0 * D);
        uint32_t oa[P::PA], ob[P::PB];
#pragma unroll
        for (int i = 0; i < P::PA; ++i) {
            const int q = i * P::threads + tid;
            oa[i] = 2u * ((uint32_t)least(P::row_of(q), m.T - 1 - t0) * D + P::k_of(q));
        }
#pragma unroll
        for (int i = 0; i < P::PB; ++i) {
            const int q = i * P::threads + tid;
            // n_of is a multiple of 8, as is N
            ob[i] = NN ? 2u * ((uint32_t)P::kn_of(q) * N + least(P::n_of(q), N - 8 - n0))
                       : 2u * ((uint32_t)least(P::row_of(q), N - 1 - n0) * D + P::k_of(q));
        }
        p.run(lds, D / BK, [&](char *buf, int i) {
            P::fetch(buf, i, [&](int i) { return ba + oa[i]; }, [&](int i) { return bb + ob[i]; });
        }, [&] {
            ba += BK * 2;
            bb += NN ? (int64_t)BK * 2 * N : BK * 2;
        });
    }
    if (D % BK) {
        const int k0 = D / BK * BK, left = D - k0;
        p.run_filled(
            lds,
            [&](int i) {
                const int q = i * P::threads + tid, k = P::k_of(q);
                return k < left ? ld16(src + (int64_t)least(t0 + P::row_of(q), m.T - 1) * D + k0 + k)
                                : zero4();
            },
            [&](int i) {
                const int q = i * P::threads + tid, k = NN ? P::kn_of(q) : P::k_of(q);
                if (k >= left)
                    return zero4();
                return NN ? ld16(weight + (int64_t)(k0 + k) * N + least(n0 + P::n_of(q), N - 8))
                          : ld16(weight + (int64_t)least(n0 + P::row_of(q), N - 1) * D + k0 + k);
            });
    }
#pragma unroll
    for (int i = 0; i < P::TI; ++i) {
        const int row = wm * (BM / WM) + i * 16 + (lane & 15), t = t0 + row;
#pragma unroll
        for (int j = 0; j < P::TJ; ++j) {
            const int c = n0 + wn * (BN / WN) + j * 16;
            f32x4 v = p.acc[i][j];
            if (apart)
                v += adapters_apart<NN>(m, list, cols / m.rp, du + (int64_t)row * m.LW, t, ad, N, c, lane);
            const int n = c + (lane >> 4) * 4;
            if (t < m.T && n < N)
                *reinterpret_cast<u32x2 *>(out + (int64_t)t * N + n) =
                    u32x2{pack_bf16_any(v[0], v[1]), pack_bf16_any(v[2], v[3])};
        }
    }
}

// ---------------------------------------------------------------- grads
// dA[e][j][h] = sum_t V[t][e, j] x[t][h]  (OUTER = false: big = x, N = H)
// dB[e][o][j] = sum_t d[t][o] U[t][e, j]  (OUTER = true: big = d, N = O)
// A block takes 128 columns of `big` and G = 128 / rp adapters with consecutive
// ids, over the tiles of its split that name one of them; both operands lie
// across and are read transposed.  64 tokens at a time, the next ones' loads in
// flight over the MFMAs of the present ones.  The two parts of the dense matrix
// are two steps over one fragment of `big`.  With one split the result is
// rounded and stored, else fp32 sums go to `part` (laid out like the result)
// to be added.
constexpr int kGradCols = 128;
constexpr int kGradBytes = BK * kGradCols * 2;
constexpr int kGradWindow = 64;
struct GradJob {
    const uint16_t *big, *dense;
    uint16_t *out;
    float *part;
    int N, splits, chunks;      // columns, splits of the tiles, blocks of 128 columns
};
template <bool OUTER>
__device__ __forceinline__ void adapter_grads(const Tiles &m, const GradJob &g, int ntile, int block, char *lds,
                                              int32_t *places)
{
    const int G = kGradCols / m.rp, N = g.N;
    const int n0 = block % g.chunks * kGradCols;
    const int split = block / g.chunks % g.splits, e0 = block / g.chunks / g.splits * G;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wb = wave >> 1, wd = wave & 1;        // the wave's half of the big columns, of the dense ones
    const int i0 = (int)((int64_t)ntile * split / g.splits);
    const int i1 = (int)((int64_t)ntile * (split + 1) / g.splits);
    const int members = least(G, m.E - e0);
    f32x4 acc[4][4];        // [big unit][dense unit]
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int d = 0; d < 4; ++d)
            acc[b][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // the next tile from `tile` on that names one of the adapters; their places
    // come in windows of kGradWindow tiles (one by one, a miss each: 3 us more of
    // 27 at 1001 tokens, 32 adapters)
    int window = i0 - kGradWindow;
    auto next_tile = [&](int tile) {
        for (; tile < i1; ++tile) {
            if (tile >= window + kGradWindow) {
                __syncthreads();
                window = tile;
                for (int q = tid; q < kGradWindow * G; q += 256) {
                    const int at = tile + q / G;
                    places[q] = at < i1 && q % G < members ? m.place[(int64_t)at * m.E + e0 + q % G] : -1;
                }
                __syncthreads();
            }
            int any = -1;
            for (int q = 0; q < members; ++q)
                any = any < places[(tile - window) * G + q] ? places[(tile - window) * G + q] : any;
            if (any >= 0)
                break;
        }
        return tile;
    };
    u32x4 rb[4], rd[4], rl[4];
    int my_at = -1;         // dense columns of the thread's pieces, -1 if not in this tile's list
    auto load_at = [&](int tile) {
        const int c = tid % 16 * 8, q = c / m.rp;
        const int p = q < members ? places[(tile - window) * G + q] : -1;
        my_at = p >= 0 ? p * m.rp + c % m.rp : -1;
    };
    auto load = [&](int tile, int r0) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int q = p * 256 + tid, row = r0 + q / 16, c = (q % 16) * 8;
            const int64_t t = (int64_t)tile * m.BM + row;
            rb[p] = t < m.T && n0 + c < N ? ld16(g.big + t * N + n0 + c) : zero4();
            rd[p] = t < m.T && my_at >= 0 ? ld16(g.dense + t * m.LW + my_at) : zero4();
        }
    };
    auto load_low = [&](int tile, int r0) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int64_t t = (int64_t)tile * m.BM + r0 + (p * 256 + tid) / 16;
            rl[p] = t < m.T && my_at >= 0 ? ld16(g.dense + m.low + t * m.LW + my_at) : zero4();
        }
    };
    int tile = next_tile(i0), r0 = 0, buf = 0;
    if (tile < i1) {
        load_at(tile);
        load(tile, 0);
        load_low(tile, 0);
    }
    // which of the wave's units the present tile has, and the next one
    bool on[4] = {false, false, false, false}, next_on[4];
    auto load_on = [&](int tile) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int q = (wd * 4 + d) * 16 / m.rp;
            next_on[d] = q < members && places[(tile - window) * G + q] >= 0;
        }
    };
    if (tile < i1)
        load_on(tile);
    // LDS: two buffers of `big`, by turns, then the upper and the lower part
    char *const l_hi = lds + 2 * kGradBytes, *const l_lo = l_hi + kGradBytes;
    auto put = [&](char *to, const u32x4 (&v)[4]) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int q = p * 256 + tid, k = q / 16, c = q % 16;
            *reinterpret_cast<u32x4 *>(to + off_n(k, c >> 1) + (c & 1) * 16) = v[p];
        }
    };
    while (tile < i1) {
        char *lb = lds + buf * kGradBytes;
        put(lb, rb);
        put(l_hi, rd);
        if (r0 == 0)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                on[d] = next_on[d];
        int tile2 = tile, r2 = r0 + BK;
        if (r2 >= m.BM || (int64_t)tile * m.BM + r2 >= m.T) {
            tile2 = next_tile(tile + 1);
            r2 = 0;
            if (tile2 < i1) {
                load_at(tile2);
                load_on(tile2);
            }
        }
        if (tile2 < i1)
            load(tile2, r2);
        __syncthreads();
        bf16x8 fb0[4], fb1[4];
        auto multiply = [&](const char *ld, int ks, const bf16x8 (&fb)[4]) {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if (!on[d])
                    continue;
                const bf16x8 fd = frag_n(ld, ks, at_n(wd * 4 + d, lane));
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    acc[b][d] = OUTER ? mfma(fd, fb[b], acc[b][d]) : mfma(fb[b], fd, acc[b][d]);
            }
        };
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            fb0[b] = frag_n(lb, 0, at_n(wb * 4 + b, lane));
            fb1[b] = frag_n(lb, 1, at_n(wb * 4 + b, lane));
        }
        multiply(l_hi, 0, fb0);
        multiply(l_hi, 1, fb1);
        // one barrier a step: what a step writes was read two steps ago at the
        // latest (`big` by turns, the upper and the lower part one step each)
        put(l_lo, rl);
        if (tile2 < i1)
            load_low(tile2, r2);
        __syncthreads();
        multiply(l_lo, 0, fb0);
        multiply(l_lo, 1, fb1);
        tile = tile2;
        r0 = r2;
        buf ^= 1;
    }
    float s = 0.0f;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                s = fmaf(acc[b][d][q], 0.0f, s);
    const bool again = __any(!(s == 0.0f));
    const int64_t total = (int64_t)m.E * m.r * N;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            // the four results of a lane: dense columns dn + (OUTER ? q : 0),
            // big columns bn + (OUTER ? 0 : q)
            const int dn = (wd * 4 + d) * 16 + (OUTER ? (lane >> 4) * 4 : (lane & 15));
            const int bn = n0 + (wb * 4 + b) * 16 + (OUTER ? (lane & 15) : (lane >> 4) * 4);
            const int j = dn % m.rp, e = e0 + dn / m.rp;
            if (dn / m.rp >= members || j >= m.r || bn >= N)
                continue;
            f32x4 v = acc[b][d];
            if (again) {
                // again, over the tokens that name the adapter only
                v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                for (int tile = i0; tile < i1; ++tile) {
                    const int l = m.place[(int64_t)tile * m.E + e];
                    for (int row = 0; l >= 0 && row < m.BM; ++row) {
                        const int64_t t = (int64_t)tile * m.BM + row;
                        bool named = false;
                        if (t < m.T)
                            for (int k = 0; k < m.K; ++k)
                                named = named || m.idx[t * m.K + k] == e;
                        if (!named)
                            continue;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            // both parts in one factor (exact): an infinity times each
                            // alone could be two of opposite signs
                            const uint16_t x = g.big[t * N + bn + (OUTER ? 0 : q)];
                            const uint16_t *y = g.dense + t * m.LW + l * m.rp + j + (OUTER ? q : 0);
                            v[q] = fmaf(bf16_lo(x), bf16_lo(*y) + bf16_lo(y[m.low]), v[q]);
                        }
                    }
                }
            }
            const int64_t o = OUTER ? ((int64_t)e * N + bn) * m.r + j : ((int64_t)e * m.r + j) * N + bn;
            if (g.splits > 1)
                *reinterpret_cast<f32x4 *>(g.part + split * total + o) = v;
            else
                *reinterpret_cast<u32x2 *>(g.out + o) =
                    u32x2{pack_bf16_any(v[0], v[1]), pack_bf16_any(v[2], v[3])};
        }
    }
}
// Both gradients in one launch: `blocks_a` blocks of dA's, the rest dB's.
__global__ void __launch_bounds__(256, 2)
adapter_grads_kernel(Tiles m, GradJob a, GradJob b, int ntile, int blocks_a)
{
    __shared__ __attribute__((aligned(16))) char lds[4 * kGradBytes];
    __shared__ int32_t places[kGradWindow * kGradCols / 16];
    if ((int)blockIdx.x < blocks_a)
        adapter_grads<false>(m, a, ntile, blockIdx.x, lds, places);
    else
        adapter_grads<true>(m, b, ntile, blockIdx.x - blocks_a, lds, places);
}

// The splits' sums, in split order, rounded to bf16: of dA's values, then dB's.
__global__ void __launch_bounds__(256)
adapter_grads_sum_kernel(GradJob a, int64_t total_a, GradJob b, int64_t total_b)
{
    const int64_t step = (int64_t)gridDim.x * 256 * 4;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < total_a + total_b; i += step) {
        const bool in_a = i < total_a;
        const GradJob &g = in_a ? a : b;
        const int64_t total = in_a ? total_a : total_b, o = in_a ? i : i - total_a;
        f32x4 v = *reinterpret_cast<const f32x4 *>(g.part + o);
#pragma unroll 4
        for (int z = 1; z < g.splits; ++z)
            v += *reinterpret_cast<const f32x4 *>(g.part + z * total + o);
        *reinterpret_cast<u32x2 *>(g.out + o) = u32x2{pack_bf16_any(v[0], v[1]), pack_bf16_any(v[2], v[3])};
    }
}

// ---------------------------------------------------------------- a few tokens
// Up to kSmallTokens tokens (a decode batch) are bound by the weights' bytes:
// every block then reads a piece of W, or of an entry's A, and nothing waits
// for a list.  One launch computes both (one token, 4096 x 4096: 5.1 us, 6.6 TB/s,
// W from the cache; 128 tokens with an adapter each, 7168 x 4096: 22 us for
// 87 MB, 4 TB/s),
//   part_w[split][t][o] = the split's share of W x_t       (MFMA, all tokens in one tile)
//   part_u[split][t, k][j] = the split's share of A_e x_t   (one entry per block)
// and a second adds the splits and B_e u, in fp32 throughout.
template <typename P>
__global__ void __launch_bounds__(256, 2)
adapter_small_kernel(const uint16_t *__restrict__ x, int T, int H,
                     const uint16_t *__restrict__ weight, int O, const uint16_t *__restrict__ a,
                     int E, int r, const int32_t *__restrict__ idx, int nb, int splits, int usplits,
                     float *__restrict__ part_w, float *__restrict__ part_u, int entries)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    static_assert(P::threads == 256, "one block shape for both parts");
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    if ((int)blockIdx.x >= nb * splits) {
        const int id = blockIdx.x - nb * splits;
        const int entry = id % entries, split = id / entries;
        const int K = entries / T, e = idx[entry];
        if ((unsigned)e >= (unsigned)E)
            return;
        // runs of 512 channels, a lane 8 of each
        const int runs = (H + 511) / 512;
        const int h0 = (int)((int64_t)runs * split / usplits) * 512;
        const int h1 = least((int)((int64_t)runs * (split + 1) / usplits) * 512, H);
        const uint16_t *xr = x + (int64_t)(entry / K) * H;
        for (int j = wave * 2; j < r; j += 8) {
            const uint16_t *a0 = a + ((int64_t)e * r + j) * H, *a1 = a0 + H;
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
            for (int h = h0 + lane * 8; h < h1; h += 512) {
                const u32x4 vx = ld16(xr + h), v0 = ld16(a0 + h), v1 = ld16(a1 + h);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    s0 = fmaf(bf16_lo(vx[q]), bf16_lo(v0[q]), s0);
                    s0 = fmaf(bf16_hi(vx[q]), bf16_hi(v0[q]), s0);
                    s1 = fmaf(bf16_lo(vx[q]), bf16_lo(v1[q]), s1);
                    s1 = fmaf(bf16_hi(vx[q]), bf16_hi(v1[q]), s1);
                }
            }
            s0 = wave_sum_f(s0);
            s1 = wave_sum_f(s1);
            if (lane < 2)
                part_u[((int64_t)split * entries + entry) * r + j + lane] = lane ? s1 : s0;
        }
        return;
    }
    const int n0 = blockIdx.x % nb * P::BN, split = blockIdx.x / nb;
    const int stages = (H + BK - 1) / BK;
    const int s0 = (int)((int64_t)stages * split / splits);
    const int s1 = (int)((int64_t)stages * (split + 1) / splits);
    const int whole = least(s1, H / BK) - s0;
    P p;
    p.zero();
    const char *ba = reinterpret_cast<const char *>(x + s0 * BK);
    const char *bb = reinterpret_cast<const char *>(weight + (int64_t)n0 * H + s0 * BK);
    uint32_t oa[P::PA], ob[P::PB];
#pragma unroll
    for (int i = 0; i < P::PA; ++i) {
        const int q = i * P::threads + tid;
        oa[i] = 2u * ((uint32_t)least(P::row_of(q), T - 1) * H + P::k_of(q));
    }
#pragma unroll
    for (int i = 0; i < P::PB; ++i) {
        const int q = i * P::threads + tid;
        ob[i] = 2u * ((uint32_t)least(P::row_of(q), O - 1 - n0) * H + P::k_of(q));
    }
    p.run(lds, whole, [&](char *buf, int i) {
        P::fetch(buf, i, [&](int i) { return ba + oa[i]; }, [&](int i) { return bb + ob[i]; });
    }, [&] {
        ba += BK * 2;
        bb += BK * 2;
    });
    if (whole < s1 - s0) {
        const int k0 = (s0 + whole) * BK, left = H - k0;
        p.run_filled(
            lds,
            [&](int i) {
                const int q = i * P::threads + tid, k = P::k_of(q);
                return k < left ? ld16(x + (int64_t)least(P::row_of(q), T - 1) * H + k0 + k) : zero4();
            },
            [&](int i) {
                const int q = i * P::threads + tid, k = P::k_of(q);
                return k < left ? ld16(weight + (int64_t)least(n0 + P::row_of(q), O - 1) * H + k0 + k)
                                : zero4();
            });
    }
    const int wm = wave / P::WN, wn = wave % P::WN;
#pragma unroll
    for (int i = 0; i < P::TI; ++i) {
        const int t = wm * (P::BM / P::WM) + i * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < P::TJ; ++j) {
            const int n = n0 + wn * (P::BN / P::WN) + j * 16 + (lane >> 4) * 4;
            if (t < T && n < O)
                *reinterpret_cast<f32x4 *>(part_w + ((int64_t)split * T + t) * O + n) = p.acc[i][j];
        }
    }
}

// out[t][o .. o+3] per thread; the token's u, times its coefficients, in
// shared memory.  W's splits are asked for first, to be there with u.
constexpr int kSmallSumThreads = 128;
__global__ void __launch_bounds__(kSmallSumThreads)
adapter_small_sum_kernel(const float *__restrict__ part_w, int splits, const float *__restrict__ part_u,
                         int usplits, int T, int O, const uint16_t *__restrict__ b, int E, int r,
                         const int32_t *__restrict__ idx, const float *__restrict__ w, int K,
                         float scale, uint16_t *__restrict__ out, int32_t *__restrict__ num_invalid)
{
    extern __shared__ float u[];        // [K, r]
    const int tid = threadIdx.x, t = blockIdx.y;
    const int32_t *row = idx + (int64_t)t * K;
    const int o = (blockIdx.x * kSmallSumThreads + tid) * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (o < O) {
        const float *p = part_w + (int64_t)t * O + o;
#pragma unroll 8
        for (int q = 0; q < splits; ++q)
            v += *reinterpret_cast<const f32x4 *>(p + (int64_t)q * T * O);
    }
    for (int i = tid; i < K * r; i += kSmallSumThreads) {
        const int k = i / r;
        float s = 0.0f;
        if ((unsigned)row[k] < (unsigned)E) {
            const float c = scale * (w ? w[(int64_t)t * K + k] : 1.0f);
            const float *p = part_u + (int64_t)t * K * r + i;
#pragma unroll 8
            for (int q = 0; q < usplits; ++q)
                s += p[(int64_t)q * T * K * r];
            s *= c;
        }
        u[i] = s;
    }
    __syncthreads();
    if (o < O) {
        for (int k = 0; k < K; ++k) {
            const int e = row[k];
            if ((unsigned)e >= (unsigned)E)
                continue;
            const uint16_t *be = b + ((int64_t)e * O + o) * r;
#pragma unroll 2
            for (int j = 0; j < r; j += 8) {
                const float *uj = u + k * r + j;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const u32x4 bv = ld16(be + c * r + j);
                    float s = 0.0f;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        s = fmaf(bf16_lo(bv[d]), uj[2 * d], s);
                        s = fmaf(bf16_hi(bv[d]), uj[2 * d + 1], s);
                    }
                    v[c] += s;
                }
            }
        }
        *reinterpret_cast<u32x2 *>(out + (int64_t)t * O + o) =
            u32x2{pack_bf16_any(v[0], v[1]), pack_bf16_any(v[2], v[3])};
    }
    if (blockIdx.x == 0 && t == 0 && tid < kWave) {
        int n = 0;
        for (int i = tid; i < T * K; i += kWave)
            n += (unsigned)idx[i] >= (unsigned)E && idx[i] != -1;
        n = wave_sum(n);
        if (tid == 0)
            num_invalid[0] = n;
    }
}

Tiles make_tiles(const AdapterPlan &p, const int32_t *idx, char *state)
{
    Tiles m{};
    m.T = p.T;
    m.K = p.K;
    m.E = p.E;
    m.r = p.r;
    m.rp = p.rp;
    m.BM = p.BM;
    m.Lmax = p.Lmax;
    m.LW = p.LW;
    m.low = (int64_t)p.ntile * p.BM * p.LW;
    m.idx = idx;
    m.cnt = reinterpret_cast<int32_t *>(state + p.off_cnt);
    m.bad = m.cnt + p.ntile;
    m.list = reinterpret_cast<int32_t *>(state + p.off_list);
    m.place = reinterpret_cast<int32_t *>(state + p.off_place);
    return m;
}

// More than 64 KB of shared memory need the attribute.
template <typename F>
hipError_t allow_lds(F *kernel, int bytes)
{
    if (bytes <= 64 * 1024)
        return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int RB, bool NN>
hipError_t shrink(const AdapterPlan &p, const Tiles &m, const uint16_t *src, const uint16_t *ad,
                  int D, float *part, hipStream_t s)
{
    const int lds_bytes = Shrink<RB, NN>::lds_bytes + p.Lmax * 4;
    const hipError_t e = allow_lds(adapter_shrink_kernel<RB, NN>, lds_bytes);
    if (e != hipSuccess)
        return e;
    adapter_shrink_kernel<RB, NN><<<p.ntile * (p.BM / RB) * p.slots, RB * 2, lds_bytes, s>>>(
        m, src, ad, D, p.slots, part);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int NS, bool NN>
hipError_t project(const AdapterPlan &p, const Tiles &m, const uint16_t *src, int D,
                   const uint16_t *weight, int N, const uint16_t *ad, const uint16_t *dense,
                   uint16_t *out, hipStream_t s)
{
    typedef Product<BM, BN, WM, WN, NS, NN> P;
    const int lds_bytes = P::lds_bytes + p.Lmax * 4;
    const hipError_t e = allow_lds(adapter_project_kernel<P, NN>, lds_bytes);
    if (e != hipSuccess)
        return e;
    adapter_project_kernel<P, NN><<<p.ntile * ((N + BN - 1) / BN), P::threads, lds_bytes, s>>>(
        m, src, D, weight, N, ad, dense, p.ntile, out);
    return hipGetLastError();
}

template <int BM, int WM, int WN>
hipError_t small(const AdapterPlan &p, const uint16_t *x, const uint16_t *weight, const uint16_t *a,
                 const int32_t *idx, float *part_w, float *part_u, hipStream_t s)
{
    typedef Product<BM, 64, WM, WN, 3, false> P;
    const hipError_t e = allow_lds(adapter_small_kernel<P>, P::lds_bytes);
    if (e != hipSuccess)
        return e;
    const int nb = (p.O + 63) / 64;
    adapter_small_kernel<P><<<nb * p.wsplits + p.T * p.K * p.usplits, 256, P::lds_bytes, s>>>(
        x, p.T, p.H, weight, p.O, a, p.E, p.r, idx, nb, p.wsplits, p.usplits, part_w, part_u, p.T * p.K);
    return hipGetLastError();
}

// shrink + gather of one direction, and its project.
template <bool NN>
hipError_t gather(const AdapterPlan &p, const Tiles &m, const uint16_t *src, int D,
                  const uint16_t *shrinker, const float *w, float scale, float *part, float *sums,
                  uint16_t *dense, const float *u, float *dw, int32_t *num_invalid, hipStream_t s)
{
    hipError_t e = p.BM == 64 ? shrink<64, NN>(p, m, src, shrinker, D, part, s)
                              : shrink<128, NN>(p, m, src, shrinker, D, part, s);
    if (e != hipSuccess)
        return e;
    adapter_gather_kernel<<<p.ntile * (p.BM / kGatherRows), 256, 0, s>>>(
        m, w, scale, p.slots, shrink_depth(D), part, sums, dense,
        u, dw, p.ntile, num_invalid);
    return hipGetLastError();
}

template <bool NN>
hipError_t project_any(const AdapterPlan &p, const Tiles &m, const uint16_t *src, int D,
                       const uint16_t *weight, int N, const uint16_t *ad, const uint16_t *dense,
                       uint16_t *out, hipStream_t s)
{
    switch (p.BM) {
    case 64:
        switch (adapter_tile_columns(p, N, NN)) {
        case 64:
            return project<64, 64, 2, 2, 4, NN>(p, m, src, D, weight, N, ad, dense, out, s);
        case 96:
            if constexpr (!NN)
                return project<64, 96, 2, 2, 4, NN>(p, m, src, D, weight, N, ad, dense, out, s);
        }
        return project<64, 128, NN ? 2 : 1, NN ? 2 : 4, 3, NN>(p, m, src, D, weight, N, ad, dense, out, s);
    case 128:
        return project<128, 128, 2, 2, 2, NN>(p, m, src, D, weight, N, ad, dense, out, s);
    }
    return project<256, 256, 2, 4, 2, NN>(p, m, src, D, weight, N, ad, dense, out, s);
}

// dA and dB; either may be left out.
hipError_t grads(const AdapterPlan &p, const Tiles &m, const uint16_t *x, const uint16_t *d_out,
                 const uint16_t *u, const uint16_t *v, uint16_t *da, uint16_t *db, float *part,
                 hipStream_t s)
{
    const int groups = (p.E + kGradCols / p.rp - 1) / (kGradCols / p.rp);
    auto job = [&](const uint16_t *big, const uint16_t *dense, uint16_t *out, int N, float *sums) {
        return GradJob{big, dense, out, sums, N, adapter_grad_splits(p, N), (N + kGradCols - 1) / kGradCols};
    };
    const int64_t elems_a = (int64_t)p.E * p.r * p.H, elems_b = (int64_t)p.E * p.r * p.O;
    const GradJob a = job(x, v, da, p.H, part);
    const GradJob b = job(d_out, u, db, p.O, part + (da && a.splits > 1 ? a.splits * elems_a : 0));
    const int blocks_a = da ? a.chunks * a.splits * groups : 0;
    const int blocks_b = db ? b.chunks * b.splits * groups : 0;
    if (blocks_a + blocks_b == 0)
        return hipSuccess;
    adapter_grads_kernel<<<blocks_a + blocks_b, 256, 0, s>>>(m, a, b, p.ntile, blocks_a);
    const hipError_t e = hipGetLastError();
    const int64_t sum_a = da && a.splits > 1 ? elems_a : 0, sum_b = db && b.splits > 1 ? elems_b : 0;
    if (e != hipSuccess || sum_a + sum_b == 0)
        return e;
    const int64_t blocks = ((sum_a + sum_b) / 4 + 255) / 256;
    adapter_grads_sum_kernel<<<blocks < 4096 ? (int)blocks : 4096, 256, 0, s>>>(a, sum_a, b, sum_b);
    return hipGetLastError();
}

}  // namespace

int adapter_grad_splits(const AdapterPlan &p, int N)
{
    const int G = kGradCols / p.rp;
    const int64_t blocks = (int64_t)((N + kGradCols - 1) / kGradCols) * ((p.E + G - 1) / G);
    // a block per CU for each of the two gradients
    int64_t splits = 256 / (blocks > 0 ? blocks : 1);
    if (splits > 16)
        splits = 16;
    if (splits > p.ntile)
        splits = p.ntile;
    return splits < 1 ? 1 : (int)splits;
}

int adapter_tile_columns(const AdapterPlan &p, int N, bool across)
{
    if (p.BM > 64)
        return p.BM;
    // a CU takes in about 31 bytes a cycle (64 x 64: 16 KB a stage in 0.25 us, 64 x 128:
    // 24 KB in 0.35 us), so a tile costs its rows and columns, times the most
    // tiles a CU gets.  Tokens x outputs x inner, with 64, 96 and 128 columns: 1001 x
    // 4096 x 1032 24.4, 27.9 and 21.0 us; 960 x 1024 x 4096 16.5, 19.5 and 23.7; 1001 x
    // 1032 x 4096 with 32 adapters 26.3, 21.5 and 25.6; the gradient of x of 960 x 4096 x
    // 1024 18.5 with 64 and 15.6 with 128 (transposing reads do not divide 96 by waves)
    auto cost = [&](int cols) {
        const int64_t tiles = (int64_t)p.ntile * ((N + cols - 1) / cols);
        return (tiles + 255) / 256 * (64 + cols);
    };
    if (!across && cost(96) < cost(64) && cost(96) < cost(128))
        return 96;
    return cost(128) >= cost(64) ? 64 : 128;
}

AdapterPlan make_adapter_plan(int T, int H, int O, int E, int K, int r)
{
    AdapterPlan p{};
    p.T = T;
    p.H = H;
    p.O = O;
    p.E = E;
    p.K = K;
    p.r = r;
    p.rp = (r + 15) / 16 * 16;
    const int N = H < O ? H : O;
    auto blocks = [&](int b) { return ((int64_t)T + b - 1) / b * ((N + b - 1) / b); };
    p.BM = blocks(256) >= 192 ? 256 : (blocks(128) >= 192 ? 128 : 64);
    p.ntile = (T + p.BM - 1) / p.BM;
    const int64_t rows = T < p.BM ? T : p.BM;
    p.Lmax = (int)(rows * K < E ? (rows * K > 0 ? rows * K : 1) : E);
    p.LW = (int)(((int64_t)p.Lmax * p.rp + kDensePad - 1) / kDensePad * kDensePad);
    // two blocks per CU
    const int rb = p.BM == 64 ? 64 : 128;
    p.slots = T > 0 ? least(512 / ((T + rb - 1) / rb), 64) : 1;
    if (p.slots < 4)
        p.slots = 4;
    const size_t entries = (size_t)T * K * r * 4;
    // what shrink_splits can come to, for any list
    auto splits = [&](int D) { return (size_t)least(p.slots, shrink_depth(D)); };
    size_t off = 0;
    p.off_cnt = off;
    off = align256(off + 2 * (size_t)p.ntile * 4);
    p.off_list = off;
    off = align256(off + (size_t)p.ntile * p.Lmax * 4);
    p.off_place = off;
    off = align256(off + (size_t)p.ntile * E * 4);
    p.off_u = off;
    off = align256(off + entries);
    p.off_dense = off;
    off = align256(off + (size_t)p.ntile * p.BM * p.LW * 2 * 2);
    const size_t state = off > 256 ? off : 256;
    p.small = T > 0 && T <= kSmallTokens;
    p.off_part = 0;
    if (p.small) {
        // about two blocks per CU for W, of 4 stages at least, and as many for A x
        const int nb = (O + 63) / 64, stages = (H + BK - 1) / BK, runs = (H + 511) / 512;
        auto within = [](int v, int hi) { return v < 1 ? 1 : (v > hi ? hi : v); };
        p.wsplits = within(512 / nb, stages > 4 ? stages / 4 : 1);
        p.usplits = within(1024 / (T * K), runs);
        p.off_partw = align256((size_t)p.usplits * entries);
        p.ws_bytes = p.off_partw + align256((size_t)p.wsplits * T * O * 4);
        p.state_bytes = 256;        // the backward makes its own
    } else {
        p.ws_bytes = align256(splits(H) * entries) + 256;
        p.state_bytes = state;
    }
    // backward: the splits' sums or those of the gradients, v and V
    size_t part = (splits(O) > splits(H) ? splits(O) : splits(H)) * entries;
    size_t both = 0;
    for (const int n : {H, O}) {
        const int z = adapter_grad_splits(p, n);
        both += z > 1 ? (size_t)z * E * r * n * 4 : 0;
    }
    part = both > part ? both : part;
    off = align256(part);
    p.off_v = off;
    off = align256(off + entries);
    p.off_vdense = off;
    off = align256(off + (size_t)p.ntile * p.BM * p.LW * 2 * 2);
    p.off_state = off;
    p.back_bytes = off + (p.small ? state : 256);
    return p;
}

hipError_t launch_adapter(const AdapterPlan &p, const uint16_t *x, const uint16_t *weight,
                          const uint16_t *a, const uint16_t *b, const int32_t *idx, const float *w,
                          float scale, uint16_t *out, int32_t *num_invalid, char *state, char *ws,
                          hipStream_t s)
{
    if (p.T == 0) {
        adapter_zero_kernel<<<1, 1, 0, s>>>(num_invalid);
        return hipGetLastError();
    }
    float *part = reinterpret_cast<float *>(ws + p.off_part);
    if (p.small) {
        float *part_w = reinterpret_cast<float *>(ws + p.off_partw);
        const hipError_t e = p.T <= 32   ? small<32, 1, 4>(p, x, weight, a, idx, part_w, part, s)
                             : p.T <= 64 ? small<64, 2, 2>(p, x, weight, a, idx, part_w, part, s)
                                         : small<128, 4, 1>(p, x, weight, a, idx, part_w, part, s);
        if (e != hipSuccess)
            return e;
        adapter_small_sum_kernel<<<dim3((p.O / 4 + kSmallSumThreads - 1) / kSmallSumThreads, p.T),
                                   kSmallSumThreads, (size_t)p.K * p.r * 4, s>>>(part_w, p.wsplits, part, p.usplits, p.T, p.O,
                                                               b, p.E, p.r, idx, w, p.K, scale, out,
                                                               num_invalid);
        return hipGetLastError();
    }
    const Tiles m = make_tiles(p, idx, state);
    uint16_t *dense = reinterpret_cast<uint16_t *>(state + p.off_dense);
    hipError_t e = gather<false>(p, m, x, p.H, a, w, scale, part,
                                 reinterpret_cast<float *>(state + p.off_u), dense, nullptr, nullptr,
                                 num_invalid, s);
    if (e == hipSuccess)
        e = project_any<false>(p, m, x, p.H, weight, p.O, b, dense, out, s);
    return e;
}

hipError_t launch_adapter_backward(const AdapterPlan &p, const uint16_t *d_out, const uint16_t *x,
                                   const uint16_t *weight, const uint16_t *a, const uint16_t *b,
                                   const int32_t *idx, const float *w, float scale, char *state,
                                   uint16_t *dx, uint16_t *da, uint16_t *db, float *dw, char *ws,
                                   hipStream_t s)
{
    if (p.small)
        state = ws + p.off_state;
    const Tiles m = make_tiles(p, idx, state);
    float *part = reinterpret_cast<float *>(ws + p.off_part);
    float *u = reinterpret_cast<float *>(state + p.off_u);
    uint16_t *dense = reinterpret_cast<uint16_t *>(state + p.off_dense);
    uint16_t *vdense = reinterpret_cast<uint16_t *>(ws + p.off_vdense);
    hipError_t e = hipSuccess;
    if (p.small)
        e = gather<false>(p, m, x, p.H, a, w, scale, part, u, dense, nullptr, nullptr, nullptr, s);
    if (e == hipSuccess && p.T > 0)
        e = gather<true>(p, m, d_out, p.O, b, w, scale, part, reinterpret_cast<float *>(ws + p.off_v),
                         vdense, u, dw, nullptr, s);
    if (e == hipSuccess && p.T > 0 && dx)
        e = project_any<true>(p, m, d_out, p.O, weight, p.H, a, vdense, dx, s);
    if (e == hipSuccess)
        e = grads(p, m, x, d_out, dense, vdense, da, db, part, s);
    return e;
}

}  // namespace ep
