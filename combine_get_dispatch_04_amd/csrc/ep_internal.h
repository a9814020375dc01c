// ep_internal.h -- host-side plans and launchers shared by the libep sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ep_common.h"

namespace ep {

// How the layout splits topk_idx: blocks ("chunks") of CT whole tokens.
// Inside a chunk, `waves` waves each take a contiguous run of entries.
struct LayoutPlan {
    int T, K, E, R;
    int CT;        // tokens per chunk
    int CE;        // entries per chunk when a row is longer than a chunk (rows
                   // then span chunks), else 0
    int nchunk;    // ceil(T / CT)
    int waves;     // waves per chunk block
    int epl;       // entries per lane (1..32, a power of two)
    int nbits;     // bits needed for an expert id in [0, E)
    // rank keys (the sender pack): E counts ranks, the entries hold experts
    // in [0, key_experts), key_div per rank; key_div == 0 for expert keys
    int key_experts, key_div;
    size_t lds;    // dynamic shared memory of the chunk kernel
    // workspace carve-up (byte offsets, 256-aligned)
    // off_tamax: [T] fp32 row maxima for the per-token modes when a row spans
    // several dispatch blocks
    size_t off_hist, off_rank, off_rpart, off_ipart, off_tamax, bytes;
};

LayoutPlan make_layout_plan(int T, int K, int E, int R);

// The layout of the sender pack: rank keys over R ranks of E/R experts each,
// plus room for its invalid-entry count (off_misc) in the workspace.
struct RankPlan {
    LayoutPlan lp;
    size_t off_misc, bytes;
};
RankPlan make_rank_plan(int T, int K, int E, int R);

struct EcPlan {
    int T, E, C;
    size_t off_cnt, off_cursor, off_tmp, off_misc, bytes;
};
EcPlan make_ec_plan(int T, int E, int C);

// `rounds` > 1: that many rounds of p.T tokens side by side (topk_idx,
// is_token_in_rank and the per-round outputs consecutive), round r's tables
// at ws + r * round_bytes (a multiple of 256).
hipError_t launch_layout(const LayoutPlan &p, const int32_t *topk_idx, int32_t *counts,
                         int32_t *offsets, int32_t *tokens_per_rank, uint8_t *is_token_in_rank,
                         int32_t *num_invalid, char *ws, hipStream_t s, int rounds = 1,
                         size_t round_bytes = 0);

// Quantisation modes; the values are those of ep_quant_t.
constexpr int kQuantBf16 = 0;
constexpr int kQuantFp8G128 = 1;
constexpr int kQuantFp8Token = 2;
constexpr int kQuantInt8Token = 3;
constexpr int kQuantMxE4M3 = 4;
constexpr int kQuantMxE5M2 = 5;
constexpr int kQuantMxE2M1 = 6;

hipError_t launch_dispatch(const LayoutPlan &p, const uint16_t *x, int H, const int32_t *topk_idx,
                           const int32_t *offsets, bool padded, int cap_or_rows, int quant,
                           void *recv_x, void *recv_scales, int32_t *slot, int32_t *recv_src,
                           int32_t *num_dropped, char *ws, hipStream_t s);

// The one-launch low-latency dispatch (padded rows, ranks found in the
// kernel): each block scans the entries before its token, so it is built for
// small batches.
constexpr int kLlMaxEntries = 4096;   // T*K
constexpr int kLlMaxTopk = 64;        // one lane per (t,k)
bool ll_dispatch_fits(int T, int K, int H, int quant);
hipError_t launch_ll_dispatch(const uint16_t *x, int T, int H, const int32_t *topk_idx, int K,
                              int E, int cap, int quant, void *recv_x, void *recv_scales,
                              int32_t *slot, int32_t *recv_src, int32_t *recv_count,
                              int32_t *num_dropped, int32_t *num_invalid, hipStream_t s);

hipError_t launch_combine(const uint16_t *y, int y_rows, int H, const int32_t *slot,
                          const float *w, int T, int K, uint16_t *out, hipStream_t s);

// The combine with fp32 output rows: the receiving rank's partial sums.
hipError_t launch_combine_partial(const uint16_t *y, int y_rows, int H, const int32_t *slot,
                                  const float *w, int S, int K, float *partial, hipStream_t s);

// The sender pack (rank layout + rank_pack_kernel) and the sender's sum of
// the partials over ranks (ep_rank.hip).
hipError_t launch_rank_pack(const RankPlan &rp, const uint16_t *x, int H, const int32_t *topk_idx,
                            const float *w, int E, int R, int max_rows, int32_t *tokens_per_rank,
                            int32_t *rank_offsets, uint16_t *send_x, int32_t *send_src,
                            int32_t *send_idx, float *send_w, int32_t *pack_pos,
                            int32_t *num_dropped, char *ws, hipStream_t s);
hipError_t launch_rank_sum(const float *partial, int rows, int H, const int32_t *pack_pos, int T,
                           int R, uint16_t *out, hipStream_t s);

hipError_t launch_ec_dispatch(const EcPlan &p, const uint16_t *x, int H,
                              const int32_t *token_indices, uint16_t *recv_x, int32_t *tok_off,
                              int32_t *tok_ent, int32_t *num_invalid, char *ws, hipStream_t s);

hipError_t launch_ec_combine(const uint16_t *y, const float *w, int E, int C, int H,
                             const int32_t *tok_off, const int32_t *tok_ent, int T,
                             uint16_t *out, hipStream_t s);

// The router (ep_router.hip).  `bf16`: logits in bf16, else fp32.
constexpr int kMaxRouteTopk = 64;     // one lane per choice

struct BalancePlan {
    int T, E, S;
    int CT, nchunk;   // tokens per chunk, chunks
    int eb;           // blocks of 16 experts
    size_t off_arrived, off_part, off_parts, off_tails, bytes;
};
BalancePlan make_balance_plan(int T, int E, int S);

hipError_t launch_route(const void *logits, bool bf16, int T, int E, int K, bool sigmoid,
                        const float *bias, bool renorm, float scale, int32_t *topk_idx,
                        float *topk_w, int32_t *num_invalid, hipStream_t s);
hipError_t launch_balance(const BalancePlan &p, const void *logits, bool bf16,
                          const int32_t *topk_idx, int K, bool sigmoid, const int32_t *seq,
                          float coef, int32_t *counts, float *slope, float *loss,
                          int32_t *num_invalid, char *ws, hipStream_t s);
hipError_t launch_router_backward(const void *logits, bool bf16, int T, int E, int K, bool sigmoid,
                                  bool renorm, float scale, const int32_t *topk_idx,
                                  const float *d_w, const float *slope, const int32_t *seq, int S,
                                  const float *d_loss, void *d_logits, hipStream_t s);

// Low-rank adapters beside a shared projection (ep_adapter.hip).
constexpr int kMaxAdapterRank = 128;
constexpr int kMaxAdapterWidth = 1 << 20;   // H, O: a tile's rows span 32-bit offsets
constexpr int kMaxAdapterTopk = 64;
constexpr int kSmallTokens = 128;

struct AdapterPlan {
    int T, H, O, E, K, r;
    int rp;           // r rounded up to 16
    int BM, ntile;    // tokens per tile, tiles
    int Lmax, LW;     // adapters a tile can name, columns of its dense matrix
    int slots;        // blocks that share a tile's shrink
    bool small;       // a few tokens: two launches, no tiles
    int wsplits, usplits;   // splits of the inner dimension then, for W x and A x
    // the state kept from the forward for the backward
    size_t off_cnt, off_list, off_place, off_u, off_dense, state_bytes;
    // the workspaces of the forward (ws_bytes) and the backward (back_bytes)
    size_t off_part, off_partw, ws_bytes, off_v, off_vdense, off_state, back_bytes;
};
AdapterPlan make_adapter_plan(int T, int H, int O, int E, int K, int r);
int adapter_grad_splits(const AdapterPlan &p, int N);
// Columns of the projection's tiles of p.BM tokens: of N outputs, W read as it
// lies or across (the gradient of x).
int adapter_tile_columns(const AdapterPlan &p, int N, bool across);

hipError_t launch_adapter(const AdapterPlan &p, const uint16_t *x, const uint16_t *weight,
                          const uint16_t *a, const uint16_t *b, const int32_t *idx, const float *w,
                          float scale, uint16_t *out, int32_t *num_invalid, char *state, char *ws,
                          hipStream_t s);
hipError_t launch_adapter_backward(const AdapterPlan &p, const uint16_t *d_out, const uint16_t *x,
                                   const uint16_t *weight, const uint16_t *a, const uint16_t *b,
                                   const int32_t *idx, const float *w, float scale, char *state,
                                   uint16_t *dx, uint16_t *da, uint16_t *db, float *dw, char *ws,
                                   hipStream_t s);

// Microscaled tensors (ep_mx.hip): `mode` one of the kQuantMx* modes.
hipError_t launch_mx_quantize(const uint16_t *x, int64_t rows, int H, int mode, void *codes, uint8_t *scales,
                              hipStream_t s);
hipError_t launch_mx_dequantize(const void *codes, const uint8_t *scales, int64_t rows, int H, int mode,
                                uint16_t *out, hipStream_t s);

// The experts' products (ep_expert.hip).  Rows of expert e: [offsets[e],
// offsets[e+1]) of `rows`, or, with offsets NULL, the first counts[e] (all, if
// NULL) of the `cap` rows from e * cap on.
struct ExpertRows {
    const int32_t *offsets, *counts;
    int rows, cap, E;
};
struct ExpertIn {
    const void *x;              // rows, in bf16 or codes
    const uint8_t *x_scales;
    const uint8_t *w, *w_scales;    // [E, O, H] in MXFP4
    int O, H;
    int half;                   // O / 2 where rows o and half + o of W are needed together, else 0
};
constexpr int kExpertPlain = 0, kExpertGated = 1, kExpertGrad = 2;
struct ExpertOut {
    void *y;
    uint8_t *scales;
    const uint16_t *d;          // kExpertGrad: the gradient of the gated rows
    int width, kind, quant;     // columns of a row of y (kExpertGrad: of d; y has twice as many)
};
hipError_t launch_expert(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, int x_quant, hipStream_t s);
// dx = W^T x for bf16 rows x of O values.
hipError_t launch_expert_across(const ExpertRows &m, const ExpertIn &in, const ExpertOut &out, hipStream_t s);

// A whole layer of experts for a few tokens (ep_expert_few.hip).
constexpr int kFewTokens = 128;
struct FewPlan {
    int T, K, E, H, I;
    int most;               // experts that the tokens can name
    bool wide;              // blocks of 128 weight rows, else of 32
    int slices, slices_up;  // blocks of H, of I
    int stage_bytes;        // LDS of a block for its tokens
    int64_t lower;          // h's lower part, so many elements behind the upper one
    size_t off_arrived, off_named, off_expert, off_count, off_entry, off_coef, off_firsts, off_h, off_part, bytes;
};
// What the first launch leaves for the second: by the place of a named expert.
struct FewTables {
    unsigned *arrived;      // [slices]
    int32_t *named, *expert, *count;
    int32_t *entry;         // [most, T]
    float *coef;
    uint64_t *firsts;       // [T]
};
FewPlan make_few_plan(int T, int K, int E, int H, int I, bool fp4);
hipError_t launch_few(const FewPlan &p, const uint16_t *x, const int32_t *idx, const float *weights, const void *up,
                      const uint8_t *up_scales, const void *down, const uint8_t *down_scales, uint16_t *out,
                      int32_t *num_invalid, char *ws, hipStream_t s);

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// LDS bytes one block may take on the current device (cached per device).
int lds_limit();

// ---------------------------------------------------------------- device helpers
// What the router's and the adapters' kernels share.
// Two fp32 values to bf16, nearest even, for any input: a NaN stays one (the
// integer form in ep_common.h, for finite values, could carry its payload away).
__device__ __forceinline__ uint32_t pack_bf16_any(float lo, float hi)
{
    typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
    const b16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

constexpr float kNegInf = -__builtin_huge_valf();

// Row shifts inside 16 lanes, then the row broadcasts, as in
// wave_inclusive_scan: lane 63 ends up with all 64 lanes' value.  The order
// of the additions is fixed, so sums are the same for every run.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f(float old, float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        (int)__float_as_uint(old), (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ float wave_sum_f(float v)
{
    v += dpp_f<0x111, 0xF>(0.0f, v);
    v += dpp_f<0x112, 0xF>(0.0f, v);
    v += dpp_f<0x114, 0xF>(0.0f, v);
    v += dpp_f<0x118, 0xF>(0.0f, v);
    v += dpp_f<0x142, 0xA>(0.0f, v);
    v += dpp_f<0x143, 0xC>(0.0f, v);
    return last_lane(v);
}
__device__ __forceinline__ float wave_max_f(float v)
{
    v = fmaxf(v, dpp_f<0x111, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x112, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x114, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x118, 0xF>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x142, 0xA>(kNegInf, v));
    v = fmaxf(v, dpp_f<0x143, 0xC>(kNegInf, v));
    return last_lane(v);
}

// ---------------------------------------------------------------- tiles of a matrix product
// What the adapters' and the experts' products share.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int BK = 64;                 // inner elements per stage of bf16: two slices of 32, one MFMA each

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

__host__ __device__ __forceinline__ int least(int a, int b) { return a < b ? a : b; }

// Blocks are dealt to the 8 XCDs in turn; this gives each XCD a run of
// consecutive tiles, so that its L2 sees the operands they share.
__device__ __forceinline__ int xcd_order(int b, int n)
{
    const int each = n / 8, rest = n % 8, x = b % 8;
    return x * each + least(x, rest) + b / 8;
}

// ---------------------------------------------------------------- microscaled codes
// What a block's largest magnitude may come to, as a power of two.
constexpr int mx_top_exponent(int mode) { return mode == kQuantMxE4M3 ? 8 : (mode == kQuantMxE5M2 ? 15 : 2); }
// The e8m0 code of a block whose largest magnitude is `top`.
template <int MODE>
__device__ __forceinline__ uint32_t mx_scale_code(float top)
{
    return (uint32_t)(mx_shared_exponent(top, mx_top_exponent(MODE)) + 127);
}
// Four 8-bit codes of v * 2^-E, E + 127 = scale_code.  E is at most 127 minus the
// format's exponent, so 2^-E is a normal number.
template <int MODE>
__device__ __forceinline__ uint32_t mx8x4(float a, float b, float c, float d, uint32_t scale_code)
{
    constexpr float top = MODE == kQuantMxE4M3 ? 448.0f : 57344.0f;
    const float m = __uint_as_float((254u - scale_code) << 23);
    const float p = __builtin_amdgcn_fmed3f(a * m, -top, top), q = __builtin_amdgcn_fmed3f(b * m, -top, top);
    const float r = __builtin_amdgcn_fmed3f(c * m, -top, top), t = __builtin_amdgcn_fmed3f(d * m, -top, top);
    return MODE == kQuantMxE4M3 ? e4m3x4(p, q, r, t) : e5m2x4(p, q, r, t);
}
// Eight values as bf16.  The conversions read the exponent field of their scale
// only, and take 0 there as 2^-127.  A code times a scale has at most four
// significant bits: exact in bf16 down to its subnormals.
__device__ __forceinline__ u32x4 e2m1_bf16x8(uint32_t codes, uint32_t scale_code)
{
    const float s = __uint_as_float(scale_code << 23);
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3))};
}
template <int MODE>
__device__ __forceinline__ u32x4 mx8_bf16x8(u32x2 codes, uint32_t scale_code)
{
    const float s = __uint_as_float(scale_code << 23);
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (MODE == kQuantMxE4M3) {
            v[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], s, false));
            v[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], s, true));
        } else {
            v[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes[i], s, false));
            v[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes[i], s, true));
        }
    }
    return v;
}

}  // namespace ep
