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
// are).  Of the tiles that there are, `group` row tiles by all columns go to an
// XCD in a row, column by column.
template <int BM>
__device__ bool find_tile(const ExpertRows &m, int nb, int group, Tile &t)
{
    __shared__ int scan[17];
    __shared__ Tile found;
    const int per = (m.E + (int)blockDim.x - 1) / (int)blockDim.x;
    const int e0 = least((int)threadIdx.x * per, m.E), e1 = least(e0 + per, m.E);
    int mine = 0, first, n;
    for (int e = e0; e < e1; ++e) {
        rows_of(m, e, first, n);
        mine += (n + BM - 1) / BM;
    }
    int total;
    int before = block_exclusive_scan(mine, scan, &total);
    // 32-bit: the host bounds row tiles times columns
    if ((int64_t)blockIdx.x >= (int64_t)total * nb)
        return false;
    const int id = xcd_order(blockIdx.x, total * nb);
    const int g0 = id / (group * nb) * group, rows = least(group, total - g0), at = id - g0 * nb;
    const int slot = g0 + at % rows;
    if (slot >= before && slot < before + mine) {
        for (int e = e0; e < e1; ++e) {
            rows_of(m, e, first, n);
            const int tiles = (n + BM - 1) / BM;
            if (slot < before + tiles) {
                const int r0 = (slot - before) * BM;
                found = Tile{e, first + r0, least(BM, n - r0), at / rows};
                break;
            }
            before += tiles;
        }
    }
    __syncthreads();
    t = found;
    return true;
}

// ---------------------------------------------------------------- behind the product
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// What becomes of a wave's sums: acc[i][j] holds row i*16 + (lane & 15) of its
// TI * 16 rows, columns j*16 + (lane >> 4)*4 ..+3 of the tile's.  With a gate,
// odd j are the other half's values of j - 1.
template <int TI, int TJ>
__device__ __forceinline__ void finish(const ExpertOut &o, f32x4 (&acc)[TI][TJ], const Tile &t, int row0, int c0)
{
    const int lane = threadIdx.x & (kWave - 1), at = (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int r = row0 + i * 16 + (lane & 15);
        const bool live = r < t.n;
        const int64_t row = t.first + (live ? r : 0);
        if (o.kind == kExpertGrad) {
#pragma unroll
            for (int j = 0; j + 1 < TJ; j += 2) {
                const int c = c0 + j * 8 + at;
                if (!live || c >= o.width)
                    continue;
                const u32x2 d2 = *reinterpret_cast<const u32x2 *>(o.d + row * o.width + c);
                float dg[4], du[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float d = q & 1 ? bf16_hi(d2[q >> 1]) : bf16_lo(d2[q >> 1]);
                    const float g = acc[i][j][q], u = acc[i][j + 1][q], s = sigmoid(g);
                    dg[q] = d * u * s * (1.0f + g * (1.0f - s));
                    du[q] = d * g * s;
                }
                uint16_t *to = static_cast<uint16_t *>(o.y) + row * (2 * (int64_t)o.width) + c;
                *reinterpret_cast<u32x2 *>(to) = u32x2{pack_bf16_any(dg[0], dg[1]), pack_bf16_any(dg[2], dg[3])};
                *reinterpret_cast<u32x2 *>(to + o.width) =
                    u32x2{pack_bf16_any(du[0], du[1]), pack_bf16_any(du[2], du[3])};
            }
            continue;
        }
        // the output's columns, one fragment of 16 after the other
        const bool gated = o.kind == kExpertGated;
        f32x4 v[TJ];
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            v[j] = acc[i][j];
            if (gated && j % 2 == 1) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[j / 2][q] = acc[i][j - 1][q] * sigmoid(acc[i][j - 1][q]) * acc[i][j][q];
            }
        }
        const int frags = gated ? TJ / 2 : TJ;
        if (o.quant == kQuantBf16) {
#pragma unroll
            for (int j = 0; j < TJ; ++j) {
                const int c = c0 + j * 16 + at;
                if (j < frags && live && c < o.width)
                    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(o.y) + row * o.width + c) =
                        u32x2{pack_bf16_any(v[j][0], v[j][1]), pack_bf16_any(v[j][2], v[j][3])};
            }
            continue;
        }
        // blocks of 32 columns: two fragments, in the four lanes of a row
#pragma unroll
        for (int j = 0; j + 1 < TJ; j += 2) {
            if (j >= frags)
                continue;
            float top = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                top = fmaxf(top, fmaxf(fabsf(v[j][q]), fabsf(v[j + 1][q])));
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const int c = c0 + j * 16;
            if (!live || c >= o.width)
                continue;
            uint8_t *y = static_cast<uint8_t *>(o.y);
            uint32_t code;
            if (o.quant == kQuantMxE2M1) {
                code = mx_scale_code<kQuantMxE2M1>(top);
                const float both[8] = {v[j][0], v[j][1], v[j][2], v[j][3],
                                       v[j + 1][0], v[j + 1][1], v[j + 1][2], v[j + 1][3]};
                const uint32_t w = e2m1x8_scaled(both, code);
                uint8_t *to = y + row * (o.width / 2) + (c + at) / 2;
                *reinterpret_cast<uint16_t *>(to) = (uint16_t)w;
                *reinterpret_cast<uint16_t *>(to + 8) = (uint16_t)(w >> 16);
            } else {
                uint8_t *to = y + row * o.width + c + at;
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
                *reinterpret_cast<uint32_t *>(to) = lo;
                *reinterpret_cast<uint32_t *>(to + 16) = hi;
            }
            if (lane < 16)
                o.scales[row * (o.width / 32) + c / 32] = (uint8_t)code;
        }
    }
}

// ---------------------------------------------------------------- microscaled rows
// BM rows x BN weight rows, WM x WN waves, the inner dimension in stages of 256
// channels (two MFMAs of 128).  A stage's codes go from memory straight to LDS,
// rows of 128 bytes in 8 pieces of 16, piece c of row r in slot c ^ (r & 7), so
// that the 16 rows a fragment reads at one c spread over the banks.  8-bit codes
// have two such tiles, of 128 channels each.  What lies outside a tile's rows or
// behind the last channel is fetched as zeros (an address outside the buffer).
// The scales, 8 bytes of a row and stage, go through registers one stage ahead.
//
// A lane's operand of a 4-bit MFMA is one block of 32 channels, 32 (lane >> 4) ..;
// of an 8-bit one the channels 16 (lane >> 4) .. and 64 + 16 (lane >> 4) ..; its
// scale operand belongs to the block 32 (lane >> 4) .. in either case.
constexpr int kStage = 256;
constexpr uint32_t kNowhere = 0x80000000u;      // no buffer is larger than 2^31 bytes

template <int BM_, int BN_, int WM_, int WN_, int NS_, int FORMAT>
struct MxProduct {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
    static constexpr bool wide = FORMAT != kQuantMxE2M1;        // 8-bit rows
    static constexpr int waves = WM * WN, threads = waves * kWave;
    static constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
    static constexpr int bytes_a = BM * (wide ? 256 : 128), bytes_b = BN * 128, bytes = bytes_a + bytes_b;
    static constexpr int scale_rows = BM + BN, scale_bytes = scale_rows * 8;
    static constexpr int lds_bytes = NS * bytes + 2 * scale_bytes;
    static constexpr int CA = bytes_a / 1024 / waves, CB = bytes_b / 1024 / waves, pieces = CA + CB;
    static constexpr int SR = (scale_rows + threads - 1) / threads;
    static_assert(CA * waves * 1024 == bytes_a && CB * waves * 1024 == bytes_b, "whole pieces per wave");
    static_assert(TJ % 4 == 0, "a block of 32 gated columns is four fragments of a wave");

    f32x4 acc[TI][TJ];

    __device__ __forceinline__ static f32x4 mfma(const u32x4 &w, int ws, const u32x4 (&x)[wide ? 2 : 1], int xs, f32x4 c)
    {
        const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
        i32x8 b = {(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3], 0, 0, 0, 0};
        if constexpr (wide) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[4 + i] = (int)x[1][i];
        }
        constexpr int fmt = FORMAT == kQuantMxE2M1 ? 4 : (FORMAT == kQuantMxE4M3 ? 0 : 1);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, fmt, 0, ws, 0, xs);
    }

    __device__ __forceinline__ void run(char *lds, const ExpertIn &in, const Tile &t)
    {
        const int tid = threadIdx.x, lane = tid & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
        const int H = in.H, HB = H / 32, n = (H + kStage - 1) / kStage;
        const int row_a = wide ? H : H / 2, row_b = H / 2;      // bytes
        const uint8_t *const xa = static_cast<const uint8_t *>(in.x) + (int64_t)t.first * row_a;
        const uint8_t *const wb = in.w + (int64_t)t.e * in.O * row_b;
        const rsrc_t ra = row_rsrc(xa, t.n * row_a);
        const rsrc_t rb = row_rsrc(wb, (int)((int64_t)in.O * row_b));
        // the tile's row q of the weight, or -1
        auto weight_row = [&](int q) {
            if (in.half == 0) {
                const int r = t.block * BN + q;
                return r < in.O ? r : -1;
            }
            const int r = t.block * (BN / 2) + (q >> 5) * 16 + (q & 15);
            return r < in.half ? r + ((q >> 4) & 1) * in.half : -1;
        };
        // A lane's pieces: rows 8 apart, the same piece of each.
        const int sub = lane >> 3, piece = (lane & 7) ^ sub;
        uint32_t oa[CA], ob[CB];
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const int c = i * waves + wave, r = c % (BM / 8) * 8 + sub;
            oa[i] = r < t.n ? (uint32_t)(r * row_a + c / (BM / 8) * 128 + piece * 16) : kNowhere;
        }
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            const int r = weight_row((i * waves + wave) * 8 + sub);
            ob[i] = r >= 0 ? (uint32_t)r * row_b + piece * 16 : kNowhere;
        }
        char *const mine = lds + wave * 1024;
        auto fetch = [&](int s) {
            char *const buf = mine + s % NS * bytes;
            const int left = H - s * kStage;            // channels
            const bool whole = left >= kStage;
#pragma unroll
            for (int i = 0; i < CA; ++i) {
                const int k = wide ? (i * waves + wave) / (BM / 8) * 128 + piece * 16 : piece * 32;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(buf + i * waves * 1024), 16,
                                                         whole || k < left ? oa[i] : kNowhere,
                                                         s * (wide ? 256 : 128), 0, 0);
            }
#pragma unroll
            for (int i = 0; i < CB; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(buf + bytes_a + i * waves * 1024), 16,
                                                         whole || piece * 32 < left ? ob[i] : kNowhere, s * 128, 0, 0);
        };
        // Scales: 8 of a row and stage, 1.0 where there is none.
        const uint8_t *ps[SR];
#pragma unroll
        for (int i = 0; i < SR; ++i) {
            const int q = i * threads + tid;
            ps[i] = nullptr;
            if (q < BM) {
                if (q < t.n)
                    ps[i] = in.x_scales + (int64_t)(t.first + q) * HB;
            } else if (q < scale_rows) {
                const int r = weight_row(q - BM);
                if (r >= 0)
                    ps[i] = in.w_scales + ((int64_t)t.e * in.O + r) * HB;
            }
        }
        auto load_scales = [&](int s, uint64_t (&v)[SR]) {
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                v[i] = 0x7F7F7F7F7F7F7F7Full;
                if (!ps[i])
                    continue;
                if (s * 8 + 8 <= HB)
                    __builtin_memcpy(&v[i], ps[i] + s * 8, 8);
                else
                    for (int b = s * 8; b < HB; ++b) {
                        const int at = (b & 7) * 8;
                        v[i] = (v[i] & ~(0xFFull << at)) | ((uint64_t)ps[i][b] << at);
                    }
            }
        };
        char *const scales = lds + NS * bytes;
        auto store_scales = [&](int s, const uint64_t (&v)[SR]) {
#pragma unroll
            for (int i = 0; i < SR; ++i)
                if (i * threads + tid < scale_rows)
                    *reinterpret_cast<uint64_t *>(scales + (s & 1) * scale_bytes + (i * threads + tid) * 8) = v[i];
        };
        // Fragments.
        const int wm = wave / WN, wn = wave % WN;
        const int r16 = lane & 15, g = lane >> 4;
        const int fa = (wm * (BM / WM) + r16) * 128, fb = bytes_a + (wn * (BN / WN) + r16) * 128;
        const int slot0 = (g ^ (r16 & 7)) << 4;         // piece g; piece 4 + g is bit 6 apart
        const int sa = (wm * (BM / WM) + r16) * 8, sb = (BM + wn * (BN / WN) + r16) * 8;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        uint64_t sc[SR];
        load_scales(0, sc);
        for (int s = 0; s < NS - 1 && s < n; ++s)
            fetch(s);
        store_scales(0, sc);
        if (n > 1)
            load_scales(1, sc);
        for (int s = 0; s < n; ++s) {
            if (s + NS - 1 <= n)
                wait_and_meet<(NS - 2) * pieces>();
            else
                wait_and_meet<0>();
            if (s + 1 < n)
                store_scales(s + 1, sc);
            if (s + 2 < n)
                load_scales(s + 2, sc);
            if (s + NS - 1 < n)
                fetch(s + NS - 1);
            const char *const buf = lds + s % NS * bytes;
            const char *const sbuf = scales + (s & 1) * scale_bytes;
            u32x2 qa[TI], qb[TJ];
#pragma unroll
            for (int i = 0; i < TI; ++i)
                qa[i] = *reinterpret_cast<const u32x2 *>(sbuf + sa + i * 128);
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                qb[j] = *reinterpret_cast<const u32x2 *>(sbuf + sb + j * 128);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4 b[TJ], a[wide ? 2 : 1];
#pragma unroll
                for (int j = 0; j < TJ; ++j)
                    b[j] = ld16(buf + fb + j * 2048 + (slot0 ^ (ks * 64)));
#pragma unroll
                for (int i = 0; i < TI; ++i) {
                    if constexpr (wide) {
                        a[0] = ld16(buf + fa + ks * (BM * 128) + i * 2048 + slot0);
                        a[1] = ld16(buf + fa + ks * (BM * 128) + i * 2048 + (slot0 ^ 64));
                    } else {
                        a[0] = ld16(buf + fa + i * 2048 + (slot0 ^ (ks * 64)));
                    }
#pragma unroll
                    for (int j = 0; j < TJ; ++j)
                        acc[i][j] = mfma(b[j], (int)(qb[j][ks] >> (8 * g)), a, (int)(qa[i][ks] >> (8 * g)), acc[i][j]);
                }
            }
        }
    }
};

// ---------------------------------------------------------------- bf16 rows
// The same with rows in bf16: the weight's codes are widened to bf16 (exactly) on
// their way to LDS, and the product is one of bf16 MFMAs.  Across = false:
// y = W x, inner dimension H.  Across = true: the gradient of the rows, dx =
// W^T d, inner dimension O: the weight lies across and is read transposed.
// A stage is 64 inner elements.  The rows go from memory straight to LDS; of the
// weight each thread takes one block of 32 codes and its scale, through registers,
// one stage ahead.
template <int BM_, int BN_, int WM_, int WN_, int NS_, bool ACROSS>
struct WideProduct {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
    static constexpr int waves = WM * WN, threads = waves * kWave;
    static constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
    static constexpr int bytes_a = BM * 128, bytes_b = BN * 128, lds_bytes = NS * bytes_a + 2 * bytes_b;
    static constexpr int CA = bytes_a / 1024 / waves, PB = BN * 2 / threads;
    static_assert(CA * waves * 1024 == bytes_a && PB * threads == BN * 2, "whole pieces");
    static_assert(TJ == 4, "gated blocks of 32, and units read four at a time");

    f32x4 acc[TI][TJ];

    __device__ __forceinline__ void run(char *lds, const ExpertIn &in, const Tile &t)
    {
        const int tid = threadIdx.x, lane = tid & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
        const int D = ACROSS ? in.O : in.H, n = (D + BK - 1) / BK;
        const int HB = in.H / 32;
        const rsrc_t ra = row_rsrc(static_cast<const uint16_t *>(in.x) + (int64_t)t.first * D, t.n * D * 2);
        const int sub = lane >> 3, piece = (lane & 7) ^ sub;
        uint32_t oa[CA];
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const int r = (i * waves + wave) * 8 + sub;
            oa[i] = r < t.n ? (uint32_t)(r * D * 2 + piece * 16) : kNowhere;
        }
        char *const mine = lds + wave * 1024;
        auto fetch = [&](int s) {
            const bool there = s * BK + piece * 8 < D;
#pragma unroll
            for (int i = 0; i < CA; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(mine + s % NS * bytes_a + i * waves * 1024), 16,
                                                         there ? oa[i] : kNowhere, s * BK * 2, 0, 0);
        };
        // A thread's blocks: weight row and block of the stage, or (across) inner row
        // and block of the tile's columns.
        const uint8_t *const wb = in.w + (int64_t)t.e * in.O * (in.H / 2);
        const uint8_t *const sb = in.w_scales + (int64_t)t.e * in.O * HB;
        int row[PB], blk[PB];       // row -1: none
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int p = i * threads + tid;
            if constexpr (ACROSS) {
                row[i] = p / (BN / 32);
                blk[i] = t.block * (BN / 32) + p % (BN / 32);
                if (blk[i] >= HB)
                    row[i] = -1;
            } else {
                const int q = p >> 1;
                blk[i] = p & 1;
                if (in.half == 0) {
                    row[i] = t.block * BN + q < in.O ? t.block * BN + q : -1;
                } else {
                    const int r = t.block * (BN / 2) + (q >> 5) * 16 + (q & 15);
                    row[i] = r < in.half ? r + ((q >> 4) & 1) * in.half : -1;
                }
            }
        }
        u32x4 codes[PB];
        uint32_t sc[PB];
        auto load_w = [&](int s) {
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int r = ACROSS ? s * BK + row[i] : row[i], b = ACROSS ? blk[i] : s * 2 + blk[i];
                codes[i] = u32x4{0u, 0u, 0u, 0u};
                sc[i] = 127u;
                if (row[i] >= 0 && r < in.O && b < HB) {
                    const int64_t at = (int64_t)r * HB + b;
                    codes[i] = ld16(wb + at * 16);
                    sc[i] = sb[at];
                }
            }
        };
        char *const lb = lds + NS * bytes_a;
        auto store_w = [&](int s) {
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int p = i * threads + tid;
                char *const to = lb + (s & 1) * bytes_b;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const u32x4 v = e2m1_bf16x8(codes[i][c], sc[i]);
                    if constexpr (ACROSS)
                        *reinterpret_cast<u32x4 *>(to + off_n(p / (BN / 32), p % (BN / 32) * 2 + (c >> 1)) + (c & 1) * 16) = v;
                    else
                        *reinterpret_cast<u32x4 *>(to + off_k(p >> 1, (p & 1) * 4 + c)) = v;
                }
            }
        };
        const int wm = wave / WN, wn = wave % WN;
        const int fa = wm * (BM / WM) * 128 + at_k(0, lane);
        const int fb = ACROSS ? at_n(wn * TJ, lane) : wn * (BN / WN) * 128 + at_k(0, lane);
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        load_w(0);
        for (int s = 0; s < NS - 1 && s < n; ++s)
            fetch(s);
        store_w(0);
        if (n > 1)
            load_w(1);
        for (int s = 0; s < n; ++s) {
            if (s + NS - 1 <= n)
                wait_and_meet<(NS - 2) * CA>();
            else
                wait_and_meet<0>();
            if (s + 1 < n)
                store_w(s + 1);
            if (s + 2 < n)
                load_w(s + 2);
            if (s + NS - 1 < n)
                fetch(s + NS - 1);
            const char *const ba = lds + s % NS * bytes_a, *const bb = lb + (s & 1) * bytes_b;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bf16x8 b[TJ];
                if constexpr (ACROSS) {
                    if (ks == 0)
                        frags_n<0>(bb, fb, b);
                    else
                        frags_n<1>(bb, fb, b);
                } else {
#pragma unroll
                    for (int j = 0; j < TJ; ++j)
                        b[j] = frag_k(bb, j * 16, fb ^ (ks * 64));
                }
#pragma unroll
                for (int i = 0; i < TI; ++i) {
                    const bf16x8 a = frag_k(ba, i * 16, fa ^ (ks * 64));
#pragma unroll
                    for (int j = 0; j < TJ; ++j)
                        acc[i][j] = mfma(b[j], a, acc[i][j]);
                }
            }
        }
    }
};

template <typename P>
__global__ void __launch_bounds__(P::threads, P::BM * P::BN >= 256 * 128 ? 2 : 1)
expert_kernel(ExpertRows m, ExpertIn in, ExpertOut out, int nb, int group)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    Tile t;
    if (!find_tile<P::BM>(m, nb, group, t))
        return;
    P p;
    p.run(lds, in, t);
    const int wave = threadIdx.x / kWave, wm = wave / P::WN, wn = wave % P::WN;
    const int columns = in.half ? P::BN / 2 : P::BN;
    finish(out, p.acc, t, wm * (P::BM / P::WM), t.block * columns + wn * (columns / P::WN));
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
    if (blocks >= 1 << 22)          // a grid's threads are 32 bits
        return hipErrorInvalidValue;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(expert_kernel<P>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, P::lds_bytes);
    if (e != hipSuccess)
        return e;
    expert_kernel<P><<<(unsigned)blocks, P::threads, P::lds_bytes, s>>>(m, in, out, nb, 4);
    return hipGetLastError();
}

// An expert's rows on average: what the host knows of them.
int64_t mean_rows(const ExpertRows &m) { return (m.offsets ? m.rows : (int64_t)m.E * m.cap) / m.E; }

template <int FORMAT>
hipError_t product_mx(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, hipStream_t s)
{
    const int cover = in.half ? in.half : in.O;
    const int64_t each = mean_rows(m);
    if (each >= 160) {
        if constexpr (FORMAT == kQuantMxE2M1)
            return product<MxProduct<256, 256, 2, 4, 2, FORMAT>>(m, in, out, cover, s);
        else
            return product<MxProduct<128, 256, 2, 4, 2, FORMAT>>(m, in, out, cover, s);
    }
    if (each >= 48)
        return product<MxProduct<128, 128, 2, 2, 2, FORMAT>>(m, in, out, cover, s);
    return product<MxProduct<32, 128, 2, 2, 4, FORMAT>>(m, in, out, cover, s);
}

template <bool ACROSS>
hipError_t product_wide(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, hipStream_t s)
{
    const int cover = ACROSS ? in.H : in.half ? in.half : in.O;
    const int64_t each = mean_rows(m);
    if (each >= 160)
        return product<WideProduct<256, 256, 2, 4, 2, ACROSS>>(m, in, out, cover, s);
    if (each >= 48)
        return product<WideProduct<128, 128, 2, 2, 2, ACROSS>>(m, in, out, cover, s);
    return product<WideProduct<32, 128, 2, 2, 4, ACROSS>>(m, in, out, cover, s);
}

}  // namespace

hipError_t launch_expert(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, int x_quant, hipStream_t s)
{
    switch (x_quant) {
        case kQuantBf16: return product_wide<false>(m, in, out, s);
        case kQuantMxE4M3: return product_mx<kQuantMxE4M3>(m, in, out, s);
        case kQuantMxE5M2: return product_mx<kQuantMxE5M2>(m, in, out, s);
        default: return product_mx<kQuantMxE2M1>(m, in, out, s);
    }
}

hipError_t launch_expert_across(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, hipStream_t s)
{
    return product_wide<true>(m, in, out, s);
}

}  // namespace ep
