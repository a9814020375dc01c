// ep_expert.hip -- the experts' products on the rows of a dispatch:
//   y[r, o] = sum_h W_e[o, h] x[r, h]        for the rows r of every expert e
// with W in MXFP4 (e2m1 codes, one e8m0 scale per 32 channels) and the rows in
// MXFP4, MXFP8 or bf16; behind it, if asked for, SwiGLU over the two halves of O,
// and the result in bf16 or in microscaled codes for the next product.
#include "ep_common.h"
#include "ep_internal.h"

namespace ep {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- which rows
// An expert's rows: [first, first + n) of the buffer.  Offsets or counts that
// reach beyond it are cut off.
__device__ __forceinline__ void rows_of(const ExpertRows &m, int e, int &first, int &n)
{
    if (m.offsets) {
        const int a = m.offsets[e], b = m.offsets[e + 1];
        first = a < 0 ? 0 : least(a, m.rows);
        n = (b < 0 ? 0 : least(b, m.rows)) - first;
    } else {
        first = e * m.cap;
        n = m.counts ? least(m.counts[e], m.cap) : m.cap;
    }
    n = n < 0 ? 0 : n;
}

struct Tile {
    int e, first, n;        // the expert, the tile's first row, its rows
    int block;              // of the output's columns
};
// The block's tile.  Row tiles go by expert; the blocks behind the last one have
// none (the host knows how many there may be at most, the device how many there
// are).  Experts' last tiles of at most half the rows, which take less time, come
// after all others, for the CUs that the last full round leaves idle (bf16, 8 experts of
// 1024 rows: 901 -> 872 us for the three products of a step; MXFP4, 64 experts of 512 rows: the
// same within 1 %).  Of either kind, `group` row tiles by all columns go to an XCD in
// a row, column by column.
// Every wave finds it for itself, a lane for every 64th of the experts: no barrier (one
// of them and the table behind it in LDS took 3 % of a tile of 256 x 256).
template <int BM>
__device__ __forceinline__ bool find_tile(const ExpertRows &m, int most, int nb, int group, Tile &t)
{
    const int lane = threadIdx.x & (kWave - 1), per = (m.E + kWave - 1) / kWave;
    const int e0 = least(lane * per, m.E), e1 = least(e0 + per, m.E);
    int first, n, longs = 0, shorts = 0;
    auto last_is_short = [](int rows) { return rows > 0 && (rows - 1) % BM < BM / 2; };
#pragma unroll 4
    for (int e = e0; e < e1; ++e) {
        rows_of(m, e, first, n);
        const int s = last_is_short(n);
        longs = least(longs + (n + BM - 1) / BM - s, most);
        shorts += s;
    }
    // offsets that overlap may ask for more tiles than there are rows: the first `most`
    const int upto_longs = wave_inclusive_scan(longs, lane), upto_shorts = wave_inclusive_scan(shorts, lane);
    const int all_longs = least(__builtin_amdgcn_readlane(upto_longs, kWave - 1), most);
    const int all_shorts = least(__builtin_amdgcn_readlane(upto_shorts, kWave - 1), most - all_longs);
    // 32-bit: the host bounds row tiles times columns
    const bool is_short = (int)blockIdx.x >= all_longs * nb;
    const int block = blockIdx.x - (is_short ? all_longs * nb : 0), total = is_short ? all_shorts : all_longs;
    if (block >= total * nb)
        return false;
    const int id = xcd_order(block, total * nb);
    const int g0 = id / (group * nb) * group, rows = least(group, total - g0), at = id - g0 * nb;
    const int slot = g0 + at % rows;
    const int upto = is_short ? upto_shorts : upto_longs;
    int before = upto - (is_short ? shorts : longs), e = e0, r0 = 0;
    const bool here = slot >= before && slot < upto;
    if (here)
        for (; e < e1; ++e) {
            rows_of(m, e, first, n);
            const int tiles = (n + BM - 1) / BM, s = last_is_short(n), mine = is_short ? s : tiles - s;
            if (slot < before + mine) {
                r0 = (is_short ? tiles - 1 : slot - before) * BM;
                break;
            }
            before += mine;
        }
    // in scalar registers, for the buffers' descriptors
    const int from = __ffsll((unsigned long long)ballot(here)) - 1;
    t = Tile{__builtin_amdgcn_readlane(e, from), __builtin_amdgcn_readlane(first + r0, from),
             __builtin_amdgcn_readlane(least(BM, n - r0), from), at / rows};
    return true;
}

// ---------------------------------------------------------------- behind the product
// 1 / (1 + exp(-v)) within 2^-20 of its value, and 0 where that is below 2^-128 (v < -88.7),
// by the units' own exponential (of 2) and reciprocal, 10 instructions; what -v log2(e)
// loses to rounding is made good to first order.  From t = 128 on the exponential is
// infinite (a correction times it would be a NaN), and beyond |v| = 2.36e38 t is: no
// correction there.  The reciprocal is that of a quarter, as the unit gives no subnormals.
__device__ __forceinline__ float sigmoid(float v)
{
    constexpr float l2e = 1.44269504f, ln2 = 0.693147181f, l2e_rest = 1.92596299e-8f;
    const float t = -v * l2e, rest = fmaf(-v, l2e, -t) - v * l2e_rest;
    const float p = __builtin_amdgcn_exp2f(t), q = fabsf(t) < 128.0f ? fmaf(p, rest * ln2, p) : p;
    return 0.25f * __builtin_amdgcn_rcpf(fmaf(q, 0.25f, 0.25f));
}

// What becomes of a wave's sums: acc[i][j] holds row i*16 + (lane & 15) of its
// TI * 16 rows, columns j*16 + (lane >> 4)*4 ..+3 of the tile's.  With a gate,
// odd j are the other half's values of j - 1.  The results go by LDS (`own`, the
// wave's part of it: TI * TJ * 512 bytes), so that memory gets whole lines of a row
// and not the few bytes that a lane has of it (at 256 x 256 the stores took 13 of a
// tile's 84 thousand cycles, now 8).
template <int KIND, int BITS, int TI, int TJ>
__device__ __forceinline__ void finish_as(const ExpertOut &o, const f32x4 (&acc)[TI][TJ], const Tile &t, int row0,
                                          int c0, char *own)
{
    constexpr bool gated = KIND == kExpertGated, grad = KIND == kExpertGrad;
    const int lane = threadIdx.x & (kWave - 1), r16 = lane & 15, at = (lane >> 4) * 4;
    // pieces of 16 bytes in a row of the wave's results; piece c of row r goes to slot
    // c ^ (the row's 128-byte line, up to 8), so that 16 rows' writes spread over the banks
    constexpr int per = TJ * 16 / (gated ? 2 : 1) * BITS / 128, rows_in_line = per < 8 ? 8 / per : 1;
    constexpr int most = per < 8 ? per - 1 : 7;
    auto place = [&](int row, int byte) {
        return own + (row * per + ((byte >> 4) ^ (row / rows_in_line & most))) * 16 + (byte & 15);
    };
    // of row i * 16 + r16: i is a constant behind it
    auto put = [&](int i, int byte) { return place(r16, byte) + i * 16 * per * 16; };
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int r = row0 + i * 16 + r16;
        const bool live = r < t.n;
        const int64_t row = t.first + (live ? r : 0);
        if constexpr (grad) {
#pragma unroll
            for (int j = 0; j + 1 < TJ; j += 2) {
                const int c = c0 + j * 8 + at;
                u32x2 d2 = {0u, 0u};
                if (live && c < o.width)
                    d2 = *reinterpret_cast<const u32x2 *>(o.d + row * o.width + c);
                float dg[4], du[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float d = q & 1 ? bf16_hi(d2[q >> 1]) : bf16_lo(d2[q >> 1]);
                    const float g = acc[i][j][q], u = acc[i][j + 1][q], s = sigmoid(g);
                    // d last: d u and d g may be beyond fp32 where the results are not
                    dg[q] = s * (1.0f + g * (1.0f - s)) * u * d;
                    du[q] = g * s * d;
                }
                // to bf16, as the matrix units take them (dx is then within 2.3e-3 of its value where
                // its own rounding alone gives 1.7e-3; as two bf16 they would double the product)
                *reinterpret_cast<u32x2 *>(put(i, (j * 8 + at) * 2)) =
                    u32x2{pack_bf16_any(dg[0], dg[1]), pack_bf16_any(dg[2], dg[3])};
                *reinterpret_cast<u32x2 *>(put(i, (TJ * 8 + j * 8 + at) * 2)) =
                    u32x2{pack_bf16_any(du[0], du[1]), pack_bf16_any(du[2], du[3])};
            }
            continue;
        }
        // the output's columns, one fragment of 16 after the other
        constexpr int frags = gated ? TJ / 2 : TJ;
        f32x4 v[frags];
#pragma unroll
        for (int j = 0; j < frags; ++j) {
            v[j] = acc[i][gated ? 2 * j : j];
            if constexpr (gated) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[j][q] = v[j][q] * sigmoid(v[j][q]) * acc[i][2 * j + 1][q];
            }
        }
        if constexpr (BITS == 16) {
#pragma unroll
            for (int j = 0; j < frags; ++j)
                *reinterpret_cast<u32x2 *>(put(i, (j * 16 + at) * 2)) =
                    u32x2{pack_bf16_any(v[j][0], v[j][1]), pack_bf16_any(v[j][2], v[j][3])};
        } else {
            // blocks of 32 columns: two fragments, in the four lanes of a row
#pragma unroll
            for (int j = 0; j < frags; j += 2) {
                float top = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    top = fmaxf(top, fmaxf(fabsf(v[j][q]), fabsf(v[j + 1][q])));
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                uint32_t code;
                if constexpr (BITS == 4) {
                    code = mx_scale_code<kQuantMxE2M1>(top);
                    const float both[8] = {v[j][0], v[j][1], v[j][2], v[j][3],
                                           v[j + 1][0], v[j + 1][1], v[j + 1][2], v[j + 1][3]};
                    const uint32_t w = e2m1x8_scaled(both, code);
                    *reinterpret_cast<uint16_t *>(put(i, (j * 16 + at) / 2)) = (uint16_t)w;
                    *reinterpret_cast<uint16_t *>(put(i, (j * 16 + 16 + at) / 2)) = (uint16_t)(w >> 16);
                } else {
                    uint32_t lo, hi;
                    if (o.quant == kQuantMxE4M3) {
                        code = mx_scale_code<kQuantMxE4M3>(top);
                        lo = mx8x4<kQuantMxE4M3>(v[j][0], v[j][1], v[j][2], v[j][3], code);
                        hi = mx8x4<kQuantMxE4M3>(v[j + 1][0], v[j + 1][1], v[j + 1][2], v[j + 1][3], code);
                    } else {
                        code = mx_scale_code<kQuantMxE5M2>(top);
                        lo = mx8x4<kQuantMxE5M2>(v[j][0], v[j][1], v[j][2], v[j][3], code);
                        hi = mx8x4<kQuantMxE5M2>(v[j + 1][0], v[j + 1][1], v[j + 1][2], v[j + 1][3], code);
                    }
                    *reinterpret_cast<uint32_t *>(put(i, j * 16 + at)) = lo;
                    *reinterpret_cast<uint32_t *>(put(i, j * 16 + 16 + at)) = hi;
                }
                const int c = c0 + j * 16;
                if (live && lane < 16 && c < o.width)
                    o.scales[row * (o.width / 32) + c / 32] = (uint8_t)code;
            }
        }
    }
    // a wave's own results: its writes come before its reads, for the compiler too
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    constexpr int columns = 128 / BITS;         // of a piece
    const int64_t line = (int64_t)o.width * (grad ? 32 : BITS) / 8;
#pragma unroll 4
    for (int p = lane; p < TI * 16 * per; p += kWave) {
        const int r = p / per, piece = p % per, in_half = grad ? piece % (per > 1 ? per / 2 : 1) : piece;
        const int c = c0 + in_half * columns;
        if (row0 + r < t.n && c < o.width)
            st16(static_cast<char *>(o.y) + (t.first + row0 + r) * line + (int64_t)c * BITS / 8 +
                     (in_half == piece ? 0 : (int64_t)o.width * 2),
                 ld16(place(r, piece * 16)));
    }
}
template <int TI, int TJ>
__device__ __forceinline__ void finish(const ExpertOut &o, const f32x4 (&acc)[TI][TJ], const Tile &t, int row0, int c0,
                                       char *own)
{
    if (o.kind == kExpertGrad)
        finish_as<kExpertGrad, 16>(o, acc, t, row0, c0, own);
    else if (o.quant == kQuantBf16 && o.kind == kExpertGated)
        finish_as<kExpertGated, 16>(o, acc, t, row0, c0, own);
    else if (o.quant == kQuantBf16)
        finish_as<kExpertPlain, 16>(o, acc, t, row0, c0, own);
    else if (o.quant == kQuantMxE2M1 && o.kind == kExpertGated)
        finish_as<kExpertGated, 4>(o, acc, t, row0, c0, own);
    else if (o.quant == kQuantMxE2M1)
        finish_as<kExpertPlain, 4>(o, acc, t, row0, c0, own);
    else if (o.kind == kExpertGated)
        finish_as<kExpertGated, 8>(o, acc, t, row0, c0, own);
    else
        finish_as<kExpertPlain, 8>(o, acc, t, row0, c0, own);
}

// ---------------------------------------------------------------- a block's product
// BM rows x BN weight rows, WM x WN waves.  The inner dimension goes in stages of two
// slices, a slice one MFMA deep: 128 channels of codes, or 32 with bf16 rows.
//
//   kRowsMx*     codes by codes, with the scaled MFMAs.
//   kRowsWide    bf16 rows: the weight's codes are widened to bf16 (exactly) on their
//                way to LDS.
//   kRowsAcross  the same for the gradient of the rows, dx = W^T d: the inner
//                dimension is O, the weight lies across and is read transposed.
//
// Codes and bf16 rows go from memory straight to LDS, a slice into one of NS buffers;
// what lies outside a tile's rows or behind the last channel is fetched as zeros (an
// address outside the buffer).  A slice's row has 4 pieces of 16 bytes (8 of 8-bit
// rows), piece c of row r in slot c ^ ((r >> 1) & 3) (c ^ (r & 7)), so that the 16 rows
// a fragment reads at one place spread over the banks.  What has to be looked at on the
// way goes through registers, into one of two buffers: the scales of codes (16 bytes of a
// row, for two stages: a row's request to L2 is 64 bytes whatever it takes of them, and
// stage by stage they were a third of all requests), a weight that is widened (a block
// of 32 codes and its scale per thread and piece, a stage at a time).
//
// A lane's operand of a 4-bit MFMA is one block of 32 channels, 32 (lane >> 4) ..;
// of an 8-bit one the channels 16 (lane >> 4) .. and 64 + 16 (lane >> 4) ..; its
// scale operand belongs to the block 32 (lane >> 4) .. in either case.
//
// What bounds it: with few rows the weight's bytes, and how little of a block's time they
// stream (16 rows for each of 64 experts of 4096 x 7168, MXFP8 rows: 216 us, 4.7 TB/s of
// the 7.1 that reading alone reaches; 4 rows for each of 256: 600 us, 6.6 TB/s): 64
// experts make four rounds of blocks, by 128 x 256 tiles as by 64 x 128, each with its own
// filling and end, and row fragments without a row are multiplied too.  With many rows,
// no single thing: MXFP4 rows by 256 x 256 tiles reach 2.6 PFLOP/s (512 rows for each of
// 64 experts, 4096 x 4096 with SwiGLU: 424 us), the matrix pipes busy for a third of it (by
// count LDS's reads and writes for a slice take as long as its MFMAs); without
// its loads the main loop is 25 % shorter, without the scales 10 %, without the LDS
// reads 10 %, and a tile of 4096 channels spends 59 of its 84 thousand cycles there
// (14 to fill the buffers, 8 for the results).  Its registers are all taken: 20 bytes a lane
// lie in scratch from before the loop until behind it.  bf16 rows: 0.94 PFLOP/s (1024 rows for
// each of 8 experts, 293 us: two rounds of 256 CUs and the short last tiles), the pipes
// busy 40 %.  8-bit rows: 1.76 PFLOP/s (512 rows for each of 64 experts, 4096 x 4096: 623 us,
// where MXFP4 rows take 427) by 128 x 256 tiles, as four buffers of 256 x 256 would need more
// than a CU's LDS.
//
// The MFMAs go in TI groups of TJ, one row of fragments each; after a group the
// row's fragment of the next slice is read into the same registers, and a few of
// the loads are started, so that LDS, memory and the matrix pipes stay busy
// together.  One barrier per slice, some groups into it: every wave then holds the
// slice in registers (its buffer is free), and the next one has arrived.
constexpr int kRowsMx4 = 0, kRowsMxE4M3 = 1, kRowsMxE5M2 = 2, kRowsWide = 3, kRowsAcross = 4;
// Outside every buffer, and with a stage's offset still below 2^32: no operand of a tile
// is larger than 2^30 bytes.
constexpr uint32_t kNowhere = 0x80000000u;

template <int BM_, int BN_, int WM_, int WN_, int NS_, int KIND>
struct ExpertProduct {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
    static constexpr bool mx = KIND <= kRowsMxE5M2, wide8 = KIND == kRowsMxE4M3 || KIND == kRowsMxE5M2;
    static constexpr bool across = KIND == kRowsAcross;
    static constexpr int slice = mx ? 128 : 32, stage = 2 * slice;      // inner elements
    static constexpr int waves = WM * WN, threads = waves * kWave;
    static constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
    static constexpr int line_a = wide8 ? 128 : 64;                     // bytes of a row and slice
    static constexpr int bytes_a = BM * line_a, bytes_b = mx ? BN * 64 : 0, bytes = bytes_a + bytes_b;
    static constexpr int scale_rows = BM + BN, side_bytes = mx ? scale_rows * 16 : BN * 128;
    static constexpr int lds_bytes = NS * bytes + 2 * side_bytes;
    // loads of 1 KB a wave and slice; `pieces` of them at least
    static constexpr int KA = bytes_a / 1024, CA = (KA + waves - 1) / waves, CB = bytes_b / 1024 / waves;
    static constexpr int pieces = KA / waves + CB;
    static constexpr int SR = (scale_rows + threads - 1) / threads, PB = BN * 2 / threads;
    static_assert(KA * 1024 == bytes_a && CB * waves * 1024 == bytes_b, "whole loads");
    static_assert(mx || PB * threads == BN * 2, "whole blocks per thread");
    static_assert(TJ % 4 == 0, "a block of 32 gated columns is four fragments of a wave");
    static_assert(NS % 2 == 0, "a stage's two slices are fetched or not together");
    static constexpr int LAG = TI > 2 ? 2 : 1;      // groups in front of the barrier

    typedef u32x4 frag_a[wide8 ? 2 : 1];
    typedef uint32_t scale_set[mx ? TI + TJ : 1];
    // what goes through registers
    struct Side {
        uint64_t scales[mx ? SR : 1][2];
        u32x4 codes[mx ? 1 : PB];
        uint32_t cs[mx ? 1 : PB];
    };

    f32x4 acc[TI][TJ];

    const ExpertIn &in;
    const Tile &t;
    char *const lds;
    int n;                          // slices
    int lane, wave;
    rsrc_t ra, rb, rs;
    uint32_t oa[CA], ob[mx ? CB : PB], os[mx ? 1 : PB];
    const uint8_t *ps[mx ? SR : 1];
    int k_a, k_b;                   // a lane's first inner element of a slice in its loads

    // The tile's row q of the weight, or -1.
    __device__ __forceinline__ int weight_row(int q) const
    {
        if (in.half == 0) {
            const int r = t.block * BN + q;
            return r < in.O ? r : -1;
        }
        const int r = t.block * (BN / 2) + (q >> 5) * 16 + (q & 15);
        return r < in.half ? r + ((q >> 4) & 1) * in.half : -1;
    }

    __device__ __forceinline__ ExpertProduct(char *lds_, const ExpertIn &in_, const Tile &t_) : in(in_), t(t_), lds(lds_)
    {
        const int tid = threadIdx.x;
        lane = tid & (kWave - 1);
        wave = __builtin_amdgcn_readfirstlane(tid / kWave);
        const int D = across ? in.O : in.H, HB = in.H / 32;
        n = (D + stage - 1) / stage * 2;
        const int row_a = mx ? (wide8 ? D : D / 2) : D * 2, row_b = in.H / 2;       // bytes
        ra = row_rsrc(static_cast<const uint8_t *>(in.x) + (int64_t)t.first * row_a, t.n * row_a);
        rb = row_rsrc(in.w + (int64_t)t.e * in.O * row_b, (int)((int64_t)in.O * row_b));
        // a lane's pieces of the loads into LDS: of 16 rows by 4, or 8 rows by 8
        const int sub4 = lane >> 2, piece4 = (lane & 3) ^ ((lane >> 3) & 3);
        const int sub8 = lane >> 3, piece8 = (lane & 7) ^ sub8;
        k_a = wide8 ? piece8 * 16 : piece4 * (mx ? 32 : 8);
        k_b = piece4 * 32;
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const int c = i * waves + wave, r = wide8 ? c * 8 + sub8 : c * 16 + sub4;
            oa[i] = r < t.n ? (uint32_t)(r * row_a + (wide8 ? piece8 : piece4) * 16) : kNowhere;
        }
        if constexpr (mx) {
#pragma unroll
            for (int i = 0; i < CB; ++i) {
                const int r = weight_row((i * waves + wave) * 16 + sub4);
                ob[i] = r >= 0 ? (uint32_t)r * row_b + piece4 * 16 : kNowhere;
            }
            // rows that the tile does not have take the scales of one that exists:
            // their results are not stored
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                const int q = least(i * threads + tid, scale_rows - 1);
                if (q < BM) {
                    ps[i] = in.x_scales + (int64_t)(t.first + least(q, t.n - 1)) * HB;
                } else {
                    const int r = weight_row(q - BM);
                    ps[i] = in.w_scales + ((int64_t)t.e * in.O + (r < 0 ? 0 : r)) * HB;
                }
            }
        } else {
            rs = row_rsrc(in.w_scales + (int64_t)t.e * in.O * HB, in.O * HB);
            // a thread's blocks: weight row and block of the stage, or (across) inner row
            // and block of the tile's columns
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int p = i * threads + tid;
                int r, b;
                if constexpr (across) {
                    r = p / (BN / 32);
                    b = t.block * (BN / 32) + p % (BN / 32);
                    if (b >= HB)
                        r = -1;
                } else {
                    r = weight_row(p >> 1);
                    b = p & 1;
                }
                os[i] = r >= 0 ? (uint32_t)r * HB + b : kNowhere;
                ob[i] = r >= 0 ? os[i] * 16 : kNowhere;
            }
        }
    }

    // Starts the wave's load i of slice q into LDS.
    __device__ __forceinline__ void fetch(int q, int i)
    {
        char *const to = lds + q % NS * bytes + wave * 1024;
        const int D = across ? in.O : in.H;
        if (i < CA) {
            if (CA * waves == KA || i * waves + wave < KA)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(to + i * waves * 1024), 16,
                                                         q * slice + k_a < D ? oa[i] : kNowhere, q * line_a, 0, 0);
        } else if constexpr (mx) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(to + bytes_a + (i - CA) * waves * 1024), 16,
                                                     q * slice + k_b < D ? ob[i - CA] : kNowhere, q * 64, 0, 0);
        }
    }
    // What goes through registers, of the stages `s` (codes: 2s and 2s + 1): from memory ...
    // SHORT: rows may have less than 16 scales (and then there are no further stages).
    template <bool SHORT>
    __device__ __forceinline__ void side_load(int s, Side &v) const
    {
        const int HB = in.H / 32;
        if constexpr (mx) {
            // the row's last sixteen at most (see side_store)
            const int at = least(s * 16, HB - 16);
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                if (HB >= 16) {
                    __builtin_memcpy(v.scales[i], ps[i] + at, 16);
                    continue;
                }
                v.scales[i][0] = v.scales[i][1] = 0;
                if constexpr (SHORT) {
#pragma unroll
                    for (int b = 0; b < 15; ++b)
                        v.scales[i][b / 8] |= b < HB ? (uint64_t)ps[i][b] << (8 * (b % 8)) : 0;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int p = i * threads + threadIdx.x;
                const bool there = across ? s * stage + p / (BN / 32) < in.O : s * 2 + (p & 1) < HB;
                const int step = across ? s * stage * HB : s * 2;
                v.codes[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, there ? ob[i] : kNowhere, step * 16, 0);
                v.cs[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, there ? os[i] : kNowhere, step, 0);
            }
        }
    }
    // ... and to LDS, in `parts` parts.
    static constexpr int parts = mx ? 1 : PB * 4;
    __device__ __forceinline__ void side_store(int s, int part, const Side &v) const
    {
        char *const to = lds + NS * bytes + (s & 1) * side_bytes;
        if constexpr (mx) {
            // behind a row's last scales come zeros: the scale 2^-127, for codes that are
            // zeros as well.  (Shifted here: behind the load it would be waited for.)
            const int HB = in.H / 32, over = HB >= 16 && s * 16 > HB - 16 ? (s * 16 - (HB - 16)) * 8 : 0;
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                const int q = i * threads + threadIdx.x;
                const uint64_t lo = over >= 64 ? v.scales[i][1] >> (over - 64)
                                    : over > 0 ? v.scales[i][0] >> over | v.scales[i][1] << (64 - over)
                                               : v.scales[i][0];
                const uint64_t hi = over >= 64 ? 0 : v.scales[i][1] >> over;
                // the blocks of a stage's slices side by side, so that a lane reads its own two
                const uint32_t a = (uint32_t)lo, b = (uint32_t)(lo >> 32), c = (uint32_t)hi, d = (uint32_t)(hi >> 32);
                if (SR * threads == scale_rows || q < scale_rows)
                    *reinterpret_cast<u32x4 *>(to + q * 16) =
                        u32x4{__builtin_amdgcn_perm(b, a, 0x05010400u), __builtin_amdgcn_perm(b, a, 0x07030602u),
                              __builtin_amdgcn_perm(d, c, 0x05010400u), __builtin_amdgcn_perm(d, c, 0x07030602u)};
            }
        } else {
            const int i = part / 4, c = part % 4, p = i * threads + threadIdx.x;
            const u32x4 w = e2m1_bf16x8(v.codes[i][c], v.cs[i]);
            if constexpr (across)
                *reinterpret_cast<u32x4 *>(to + off_n(p / (BN / 32), p % (BN / 32) * 2 + (c >> 1)) + (c & 1) * 16) = w;
            else
                *reinterpret_cast<u32x4 *>(to + off_k(p >> 1, (p & 1) * 4 + c)) = w;
        }
    }

    // Fragments of slice q, the KS-th of its stage.
    __device__ __forceinline__ void read_a(frag_a &a, int q, int i) const
    {
        const char *const from = lds + q % NS * bytes + (wave / WN * (BM / WM) + i * 16 + (lane & 15)) * line_a;
        if constexpr (wide8) {
            const int slot = ((lane >> 4) ^ (lane & 7)) << 4;       // piece lane >> 4; the one 4 on is bit 6 apart
            a[0] = ld16(from + slot);
            a[1] = ld16(from + (slot ^ 64));
        } else {
            a[0] = ld16(from + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4));
        }
    }
    template <int KS>
    __device__ __forceinline__ void read_b(u32x4 (&b)[TJ], int q, int j) const
    {
        const char *const side = lds + NS * bytes + ((q >> 1) & 1) * side_bytes;
        const int row = wave % WN * (BN / WN) + j * 16 + (lane & 15);
        if constexpr (mx) {
            b[j] = ld16(lds + q % NS * bytes + bytes_a + row * 64 + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4));
        } else if constexpr (across) {
            if (j % 4 != 0)
                return;
            bf16x8 v[4];
            frags_n<KS>(side, at_n(wave % WN * TJ + j, lane), v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[j + i] = __builtin_bit_cast(u32x4, v[i]);
        } else {
            b[j] = ld16(side + row * 128 + ((((lane >> 4) ^ (lane & 7)) << 4) ^ (KS * 64)));
        }
    }
    // A lane's scales of both slices of stage s, for the wave's fragment f of the rows
    // (< TI) or the weight.
    __device__ __forceinline__ uint32_t read_scale(int s, int f) const
    {
        const int row = f < TI ? wave / WN * (BM / WM) + f * 16 : BM + wave % WN * (BN / WN) + (f - TI) * 16;
        return *reinterpret_cast<const uint16_t *>(lds + NS * bytes + ((s >> 1) & 1) * side_bytes +
                                                   (row + (lane & 15)) * 16 + (s & 1) * 8 + (lane >> 4) * 2);
    }

    template <int KS>
    __device__ __forceinline__ void group(int i, const frag_a &x, const u32x4 (&b)[TJ], const scale_set &scale)
    {
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            if constexpr (mx) {
                const i32x8 w = {(int)b[j][0], (int)b[j][1], (int)b[j][2], (int)b[j][3], 0, 0, 0, 0};
                i32x8 r = {(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3], 0, 0, 0, 0};
                if constexpr (wide8) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        r[4 + c] = (int)x[1][c];
                }
                constexpr int fmt = KIND == kRowsMx4 ? 4 : (KIND == kRowsMxE4M3 ? 0 : 1);
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, r, acc[i][j], 4, fmt, KS,
                                                                             (int)scale[TI + j], KS, (int)scale[i]);
            } else {
                acc[i][j] = mfma(__builtin_bit_cast(bf16x8, b[j]), __builtin_bit_cast(bf16x8, x[0]), acc[i][j]);
            }
        }
    }

    // Slice q, the KS-th of its stage: b holds its weight fragments, b_next takes the
    // next one's.  NEXT: there is another one; FETCH: and a slice NS on.  ROWS: the wave
    // has rows of the tile (else it only loads for the others).
    template <int KS, bool NEXT, bool FETCH, bool ROWS>
    __device__ __forceinline__ void step(int q, frag_a (&a)[TI], const u32x4 (&b)[TJ], u32x4 (&b_next)[TJ],
                                         scale_set &scale, Side &side)
    {
        if constexpr (ROWS) {
#pragma unroll
            for (int g = 0; g < (NEXT ? LAG : TI); ++g)
                group<KS>(g, a[g], b, scale);
        }
        if constexpr (!NEXT)
            return;
        if constexpr (FETCH)
            wait_and_meet<(NS - 2) * pieces>();
        else
            wait_and_meet<0>();
        constexpr int rest = TI - LAG > 0 ? TI - LAG : 1;
        constexpr int loads = CA + CB;
        constexpr int RF = (loads + rest - 1) / rest, RN = (TJ + rest - 1) / rest, RP = (parts + rest - 1) / rest;
        uint32_t next[mx ? TJ : 1];
        // the stages after the next ones; the next ones' go to LDS below.  (Behind the last
        // stage the last ones again, not used.)
        constexpr int lg = mx ? 2 : 1;          // slices of a side's stages
        const bool turn = !mx || (q & 2);
        const int sides = mx ? (n + 3) >> 2 : n >> 1;
        if (KS == 1 && turn)
            side_load<false>(least((q >> lg) + 2, sides - 1), side);
#pragma unroll
        for (int h = 0; h < rest; ++h) {
            const int g = LAG + h;
            if (ROWS && g < TI)
                group<KS>(g, a[g], b, scale);
            // not before these MFMAs, which would wait for the reads as well
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (ROWS) {
#pragma unroll
                for (int j = h * RN; j < (h + 1) * RN && j < TJ; ++j) {
                    read_b<1 - KS>(b_next, q + 1, j);
                    if constexpr (mx && KS == 1)
                        next[j] = read_scale(q / 2 + 1, TI + j);
                }
#pragma unroll
                for (int i = h == 0 ? 0 : g; i <= g && i < TI; ++i) {
                    read_a(a[i], q + 1, i);
                    if constexpr (mx && KS == 1)
                        scale[i] = read_scale(q / 2 + 1, i);
                }
            }
            if constexpr (FETCH) {
#pragma unroll
                for (int i = h * RF; i < (h + 1) * RF && i < loads; ++i)
                    fetch(q + NS, i);
            }
            if (KS == 0 && turn) {
#pragma unroll
                for (int p = h * RP; p < (h + 1) * RP && p < parts; ++p)
                    side_store((q >> lg) + 1, p, side);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (mx && KS == 1 && ROWS) {
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                scale[TI + j] = next[j];
        }
    }

    // Every wave of the block comes here, with ROWS or without: they meet at the same
    // number of barriers.
    template <bool ROWS>
    __device__ __forceinline__ void run()
    {
        if constexpr (ROWS)
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j)
                    acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        Side first, side;
#pragma unroll
        for (int i = 0; i < CA + CB; ++i)
            fetch(0, i);
        side_load<true>(0, first);
        for (int q = 1; q < NS && q < n; ++q)
#pragma unroll
            for (int i = 0; i < CA + CB; ++i)
                fetch(q, i);
        side_load<false>(least(1, (mx ? (n + 3) >> 2 : n >> 1) - 1), side);
#pragma unroll
        for (int p = 0; p < parts; ++p)
            side_store(0, p, first);
        // slice 0, and what came through registers in front of the other slices
        if (n >= NS)
            wait_and_meet<(NS - 1) * pieces>();
        else
            wait_and_meet<0>();
        frag_a a[TI];
        u32x4 b0[TJ], b1[TJ];
        scale_set scale;
        if constexpr (ROWS) {
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                read_b<0>(b0, 0, j);
#pragma unroll
            for (int i = 0; i < TI; ++i)
                read_a(a[i], 0, i);
            if constexpr (mx) {
#pragma unroll
                for (int f = 0; f < TI + TJ; ++f)
                    scale[f] = read_scale(0, f);
            }
        }
        int q = 0;
        for (; q + NS < n; q += 2) {
            step<0, true, true, ROWS>(q, a, b0, b1, scale, side);
            step<1, true, true, ROWS>(q + 1, a, b1, b0, scale, side);
        }
#pragma unroll 1
        for (; q + 2 < n; q += 2) {
            step<0, true, false, ROWS>(q, a, b0, b1, scale, side);
            step<1, true, false, ROWS>(q + 1, a, b1, b0, scale, side);
        }
        step<0, true, false, ROWS>(q, a, b0, b1, scale, side);
        step<1, false, false, ROWS>(q + 1, a, b1, b0, scale, side);
    }
};

template <typename P>
__global__ void __launch_bounds__(P::threads, P::waves / 4)
expert_kernel(ExpertRows m, ExpertIn in, ExpertOut out, int most, int nb, int group)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    Tile t;
    if (!find_tile<P::BM>(m, most, nb, group, t))
        return;
    P p(lds, in, t);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wm = wave / P::WN, wn = wave % P::WN;
    // an expert's last tile may leave the lower waves without rows: the matrix pipes are
    // then the upper ones' alone
    const bool rows = wm * (P::BM / P::WM) < t.n;
    if (rows)
        p.template run<true>();
    else
        p.template run<false>();
    const int columns = in.half ? P::BN / 2 : P::BN;
    static_assert(P::BM * P::BN * 2 <= P::lds_bytes, "a tile's results fit where its operands were");
    __syncthreads();
    if (!rows)
        return;
    finish(out, p.acc, t, wm * (P::BM / P::WM), t.block * columns + wn * (columns / P::WN),
           lds + wave * (P::TI * P::TJ * 512));
}

// Row tiles that there can be.
int64_t row_tiles(const ExpertRows &m, int BM)
{
    if (!m.offsets)
        return (int64_t)m.E * ((m.cap + BM - 1) / BM);
    const int64_t named = least(m.E, m.rows);
    return (m.rows + named * (BM - 1)) / BM;
}

// How many columns the output tiles cover: all of O, the gated half, or (across) H.
template <typename P>
hipError_t product(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, int cover, hipStream_t s)
{
    const int columns = in.half ? P::BN / 2 : P::BN;
    const int nb = (cover + columns - 1) / columns;
    const int64_t blocks = row_tiles(m, P::BM) * nb;
    if (blocks == 0)
        return hipSuccess;
    if (blocks >= 1 << 23)          // a grid's threads are 32 bits
        return hipErrorInvalidValue;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(expert_kernel<P>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, P::lds_bytes);
    if (e != hipSuccess)
        return e;
    expert_kernel<P><<<(unsigned)blocks, P::threads, P::lds_bytes, s>>>(m, in, out, (int)(blocks / nb), nb, 4);
    return hipGetLastError();
}

// The tile, by what the host knows: an expert's rows on average (of a padded buffer the
// capacity, whatever the counts: a decode batch may get a larger tile padded than
// contiguous; 16 rows for each of 64 experts take 216 us either way), and how many blocks
// there would be (a ragged end for every second expert).  Large tiles take in the
// least, small ones leave no CU idle and waste less of a short expert; the limits between
// them are simple ones, up to 8 % behind the best of a line below.  us with 256 x
// 256, 128 x 256, 128 x 128 and 64 x 128 (4096 x 4096 weights unless said):
//   MXFP4, 64 experts   512 rows each 429, 493, 517, 654     64 rows 172, 162, 157, 171
//                       16 rows (7168) 243, 206, 224, 215
//   MXFP8, 64 experts   512 rows -, 605, 798, 767            64 rows -, 180, 209, 182
//                       16 rows (7168) -, 227, 291, 224
//   bf16, and back      8 experts of 1024 rows 902, 1079, 1077, 1348
//                       12 of 167 (1120 x 1032) 63, 50, 39, 42
template <int KIND>
hipError_t product_any(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, hipStream_t s)
{
    const int cover = KIND == kRowsAcross ? in.H : in.half ? in.half : in.O;
    const int64_t each = (m.offsets ? m.rows : (int64_t)m.E * m.cap) / m.E;
    auto enough = [&](int BM, int BN) {
        const int64_t tiles = (each * m.E) / BM + (m.E + 1) / 2;
        return tiles * ((cover * (in.half ? 2 : 1) + BN - 1) / BN) >= 192;
    };
    constexpr bool mx8 = KIND == kRowsMxE4M3 || KIND == kRowsMxE5M2;
    if constexpr (!mx8) {
        if (each >= 160 && enough(256, 256))
            return product<ExpertProduct<256, 256, 2, 4, 4, KIND>>(m, in, out, cover, s);
    }
    if constexpr (KIND == kRowsWide || KIND == kRowsAcross) {
        if (each >= 48 && enough(128, 128))
            return product<ExpertProduct<128, 128, 2, 2, 4, KIND>>(m, in, out, cover, s);
    } else {
        if (each >= 48 && enough(128, 256))
            return product<ExpertProduct<128, 256, 2, 4, 4, KIND>>(m, in, out, cover, s);
    }
    return product<ExpertProduct<64, 128, 2, 2, 4, KIND>>(m, in, out, cover, s);
}

}  // namespace

hipError_t launch_expert(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, int x_quant, hipStream_t s)
{
    switch (x_quant) {
        case kQuantBf16: return product_any<kRowsWide>(m, in, out, s);
        case kQuantMxE4M3: return product_any<kRowsMxE4M3>(m, in, out, s);
        case kQuantMxE5M2: return product_any<kRowsMxE5M2>(m, in, out, s);
        default: return product_any<kRowsMx4>(m, in, out, s);
    }
}

hipError_t launch_expert_across(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, hipStream_t s)
{
    return product_any<kRowsAcross>(m, in, out, s);
}

}  // namespace ep
