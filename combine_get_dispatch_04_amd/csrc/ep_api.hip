// ep_api.hip -- the C ABI declared in include/ep.h: argument checks,
// workspace sizing, and stream-ordered launches of the gfx950 kernels.
// Every check happens before anything is enqueued, so a rejected call has
// no effect.  Nothing here touches the GPU except the launches.
#include "ep.h"

#include <hip/hip_runtime.h>

#include <mutex>

#include "ep_internal.h"

namespace {

constexpr int kMaxExperts = 4096;   // the layout keeps per-expert counts in LDS
constexpr int kMaxRanks = 1024;
constexpr int64_t kI32 = 2147483647LL;
constexpr int kMaxHidden = 1 << 24; // row byte counts and offsets stay 32-bit in the kernels

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

ep_status_t hip_status(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

ep_status_t check_layout_sizes(int T, int K, int E, int R)
{
    if (T < 0 || K < 1 || E < 1 || R < 1)
        return EP_ERR_INVALID_ARG;
    if (E > kMaxExperts || R > kMaxRanks)
        return EP_ERR_UNSUPPORTED;
    if (E % R != 0)
        return EP_ERR_INVALID_ARG;
    if ((int64_t)T * K > kI32)
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

ep_status_t check_ws(const void *ws, size_t ws_bytes, size_t need)
{
    if (!ws || !aligned(ws, 256) || ws_bytes < need)
        return EP_ERR_WORKSPACE;
    return EP_OK;
}

// The arguments of a dispatch (ep_dispatch and the no-allocation form),
// other than the workspace.
ep_status_t check_dispatch_args(const uint16_t *x, int T, int H, const int32_t *topk_idx, int K,
                                int E, const int32_t *offsets, ep_recv_layout_t layout,
                                int cap_or_max_rows, ep_quant_t quant, const void *recv_x,
                                const void *recv_scales, const int32_t *slot,
                                const int32_t *recv_src, const int32_t *num_dropped)
{
    ep_status_t st = check_layout_sizes(T, K, E, 1);
    if (st != EP_OK)
        return st;
    if (layout != EP_LAYOUT_CONTIGUOUS && layout != EP_LAYOUT_PADDED)
        return EP_ERR_INVALID_ARG;
    if ((int)quant < (int)EP_QUANT_BF16 || (int)quant > (int)EP_QUANT_MXFP4_E2M1)
        return EP_ERR_INVALID_ARG;
    const bool quantised = quant != EP_QUANT_BF16;
    const bool mx = quant == EP_QUANT_MXFP8_E4M3 || quant == EP_QUANT_MXFP8_E5M2 ||
                    quant == EP_QUANT_MXFP4_E2M1;
    const bool padded = layout == EP_LAYOUT_PADDED;
    if (H < 8 || H % 8 != 0 || (quant == EP_QUANT_FP8_E4M3_G128 && H % 128 != 0) ||
        (mx && H % 32 != 0))
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (cap_or_max_rows < 0)
        return EP_ERR_INVALID_ARG;
    const int64_t rows = padded ? (int64_t)E * cap_or_max_rows : cap_or_max_rows;
    if (rows > kI32)
        return EP_ERR_INVALID_ARG;
    if (!offsets || !num_dropped || (T > 0 && (!x || !topk_idx || !slot)) ||
        (rows > 0 && T > 0 && !recv_x) || (quantised && rows > 0 && T > 0 && !recv_scales))
        return EP_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(recv_x, 16) || (!mx && !aligned(recv_scales, 4)) ||
        !aligned(topk_idx, 4) || !aligned(offsets, 4) || !aligned(slot, 4) ||
        !aligned(recv_src, 4) || !aligned(num_dropped, 4))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// Scratch of ep_layout_dispatch_noalloc: the layout's per-chunk tables and
// per-entry ranks, which the dispatch then reads (what the workspace holds
// for the pair).  Each device holds its own copy for the life of the
// process.  Host code never passes the array's name to a kernel (on the
// host it is only a stand-in for the symbol): it uses the device address
// that hipGetSymbolAddress returned for the device, taken once per device
// with that device current.
__device__ __align__(256) char scratch[EP_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;

// The device address of `scratch` on the device that runs `stream`, or
// nullptr if the runtime cannot give it.
char *scratch_for(hipStream_t stream)
{
    static std::mutex mu;
    static void *addr[kMaxDevices] = {};
    int cur = -1, dev = -1;
    if (hipGetDevice(&cur) != hipSuccess) {
        (void)hipGetLastError();
        return nullptr;
    }
    dev = cur;
    if (stream && (hipStreamGetDevice(stream, &dev) != hipSuccess)) {
        (void)hipGetLastError();
        return nullptr;
    }
    if (dev < 0 || dev >= kMaxDevices)
        return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        if (dev != cur && hipSetDevice(dev) != hipSuccess) {
            (void)hipGetLastError();
            return nullptr;
        }
        void *p = nullptr;
        const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (dev != cur)
            (void)hipSetDevice(cur);
        if (e != hipSuccess || !p) {
            (void)hipGetLastError();
            return nullptr;
        }
        addr[dev] = p;
    }
    return static_cast<char *>(addr[dev]);
}

}  // namespace

extern "C" {

const char *ep_status_string(ep_status_t status)
{
    switch (status) {
    case EP_OK:
        return "ok";
    case EP_ERR_INVALID_ARG:
        return "invalid argument";
    case EP_ERR_UNSUPPORTED:
        return "unsupported size or mode";
    case EP_ERR_WORKSPACE:
        return "workspace missing, misaligned or too small";
    case EP_ERR_HIP:
        return "HIP launch error";
    }
    return "unknown status";
}

size_t ep_workspace_bytes(int T, int K, int E, int R)
{
    if (check_layout_sizes(T, K, E, R) != EP_OK)
        return 0;
    return ep::make_layout_plan(T, K, E, R).bytes;
}

size_t ep_ec_workspace_bytes(int T, int E, int C)
{
    if (T < 0 || E < 1 || C < 1 || (int64_t)E * C > kI32 || T >= kI32)
        return 0;
    return ep::make_ec_plan(T, E, C).bytes;
}

ep_status_t ep_get_dispatch_layout(const int32_t *topk_idx, int T, int K, int E, int R,
                                   int32_t *counts, int32_t *offsets, int32_t *tokens_per_rank,
                                   uint8_t *is_token_in_rank, int32_t *num_invalid, void *ws,
                                   size_t ws_bytes, void *stream)
{
    ep_status_t st = check_layout_sizes(T, K, E, R);
    if (st != EP_OK)
        return st;
    if ((T > 0 && !topk_idx) || !counts || !offsets || !num_invalid)
        return EP_ERR_INVALID_ARG;
    if (!aligned(topk_idx, 4) || !aligned(counts, 4) || !aligned(offsets, 4) ||
        !aligned(tokens_per_rank, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    ep::LayoutPlan p = ep::make_layout_plan(T, K, E, R);
    if ((st = check_ws(ws, ws_bytes, p.bytes)) != EP_OK)
        return st;
    return hip_status(ep::launch_layout(p, topk_idx, counts, offsets, tokens_per_rank,
                                        is_token_in_rank, num_invalid, static_cast<char *>(ws),
                                        static_cast<hipStream_t>(stream)));
}

size_t ep_workspace_bytes_rounds(int T, int K, int E, int R, int round_tokens)
{
    if (check_layout_sizes(T, K, E, R) != EP_OK || round_tokens < 1)
        return 0;
    const int rt = round_tokens < T ? round_tokens : T;
    if (rt == 0)
        return ep::make_layout_plan(0, K, E, R).bytes;
    const int full = T / rt, last = T - full * rt;
    const size_t stride = ep::make_layout_plan(rt, K, E, R).bytes;
    return stride * (size_t)full + (last ? ep::make_layout_plan(last, K, E, R).bytes : 0);
}

ep_status_t ep_get_dispatch_layout_rounds(const int32_t *topk_idx, int T, int K, int E, int R,
                                          int round_tokens, int32_t *counts, int32_t *offsets,
                                          int32_t *tokens_per_rank, uint8_t *is_token_in_rank,
                                          int32_t *num_invalid, void *ws, size_t ws_bytes,
                                          void *stream)
{
    ep_status_t st = check_layout_sizes(T, K, E, R);
    if (st != EP_OK)
        return st;
    if (round_tokens < 1)
        return EP_ERR_INVALID_ARG;
    if ((T > 0 && !topk_idx) || !counts || !offsets || !num_invalid)
        return EP_ERR_INVALID_ARG;
    if (!aligned(topk_idx, 4) || !aligned(counts, 4) || !aligned(offsets, 4) ||
        !aligned(tokens_per_rank, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, ep_workspace_bytes_rounds(T, K, E, R, round_tokens))) !=
        EP_OK)
        return st;
    if (T == 0)
        return EP_OK;                       // no rounds: nothing to write
    const int rt = round_tokens < T ? round_tokens : T;
    const int full = T / rt, last = T - full * rt;
    const ep::LayoutPlan p = ep::make_layout_plan(rt, K, E, R);
    const size_t stride = p.bytes;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    char *w = static_cast<char *>(ws);
    // the full rounds, at most 65535 per launch pair (grid.y / grid.x)
    for (int r0 = 0; r0 < full; r0 += 65535) {
        const int n = full - r0 < 65535 ? full - r0 : 65535;
        hipError_t e = ep::launch_layout(
            p, topk_idx + (int64_t)r0 * rt * K, counts + (int64_t)r0 * E,
            offsets + (int64_t)r0 * (E + 1), tokens_per_rank ? tokens_per_rank + (int64_t)r0 * R : nullptr,
            is_token_in_rank ? is_token_in_rank + (int64_t)r0 * rt * R : nullptr,
            num_invalid + r0, w + stride * (size_t)r0, s, n, stride);
        if (e != hipSuccess)
            return EP_ERR_HIP;
    }
    if (last) {
        const ep::LayoutPlan pl = ep::make_layout_plan(last, K, E, R);
        const int64_t t0 = (int64_t)full * rt;
        return hip_status(ep::launch_layout(
            pl, topk_idx + t0 * K, counts + (int64_t)full * E, offsets + (int64_t)full * (E + 1),
            tokens_per_rank ? tokens_per_rank + (int64_t)full * R : nullptr,
            is_token_in_rank ? is_token_in_rank + t0 * R : nullptr, num_invalid + full,
            w + stride * (size_t)full, s));
    }
    return EP_OK;
}

ep_status_t ep_dispatch(const uint16_t *x, int T, int H, const int32_t *topk_idx, int K, int E,
                        const int32_t *offsets, ep_recv_layout_t layout, int cap_or_max_rows,
                        ep_quant_t quant, void *recv_x, void *recv_scales, int32_t *slot,
                        int32_t *recv_src, int32_t *num_dropped, void *ws, size_t ws_bytes,
                        void *stream)
{
    ep_status_t st = check_dispatch_args(x, T, H, topk_idx, K, E, offsets, layout,
                                         cap_or_max_rows, quant, recv_x, recv_scales, slot,
                                         recv_src, num_dropped);
    if (st != EP_OK)
        return st;
    ep::LayoutPlan p = ep::make_layout_plan(T, K, E, 1);
    if ((st = check_ws(ws, ws_bytes, p.bytes)) != EP_OK)
        return st;
    return hip_status(ep::launch_dispatch(p, x, H, topk_idx, offsets,
                                          layout == EP_LAYOUT_PADDED, cap_or_max_rows,
                                          (int)quant,
                                          recv_x, recv_scales, slot, recv_src, num_dropped,
                                          static_cast<char *>(ws),
                                          static_cast<hipStream_t>(stream)));
}

ep_status_t ep_layout_dispatch_noalloc(const uint16_t *x, int T, int H, const int32_t *topk_idx,
                                       int K, int E, int R, int32_t *counts, int32_t *offsets,
                                       int32_t *tokens_per_rank, uint8_t *is_token_in_rank,
                                       int32_t *num_invalid, ep_recv_layout_t layout,
                                       int cap_or_max_rows, ep_quant_t quant, void *recv_x,
                                       void *recv_scales, int32_t *slot, int32_t *recv_src,
                                       int32_t *num_dropped, void *stream)
{
    // every check of ep_get_dispatch_layout and ep_dispatch, then the size
    // check, all before anything is enqueued
    ep_status_t st = check_layout_sizes(T, K, E, R);
    if (st != EP_OK)
        return st;
    if ((T > 0 && !topk_idx) || !counts || !offsets || !num_invalid)
        return EP_ERR_INVALID_ARG;
    if (!aligned(counts, 4) || !aligned(tokens_per_rank, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    st = check_dispatch_args(x, T, H, topk_idx, K, E, offsets, layout, cap_or_max_rows, quant,
                             recv_x, recv_scales, slot, recv_src, num_dropped);
    if (st != EP_OK)
        return st;
    const ep::LayoutPlan pl = ep::make_layout_plan(T, K, E, R);
    const ep::LayoutPlan pd = ep::make_layout_plan(T, K, E, 1);
    if (pl.bytes > EP_NOALLOC_SCRATCH_BYTES || pd.bytes > EP_NOALLOC_SCRATCH_BYTES)
        return EP_ERR_UNSUPPORTED;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = scratch_for(s);
    if (!ws)
        return EP_ERR_HIP;
    // the layout writes every table entry the dispatch reads, so the
    // scratch needs no clearing between calls
    hipError_t e = ep::launch_layout(pl, topk_idx, counts, offsets, tokens_per_rank,
                                     is_token_in_rank, num_invalid, ws, s);
    if (e != hipSuccess)
        return EP_ERR_HIP;
    return hip_status(ep::launch_dispatch(pd, x, H, topk_idx, offsets,
                                          layout == EP_LAYOUT_PADDED, cap_or_max_rows,
                                          (int)quant, recv_x, recv_scales, slot, recv_src,
                                          num_dropped, ws, s));
}

ep_status_t ep_low_latency_dispatch(const uint16_t *x, int T, int H, const int32_t *topk_idx,
                                    int K, int E, int cap, ep_quant_t quant, void *recv_x,
                                    void *recv_scales, int32_t *slot, int32_t *recv_src,
                                    int32_t *recv_count, int32_t *num_dropped,
                                    int32_t *num_invalid, void *stream)
{
    ep_status_t st = check_layout_sizes(T, K, E, 1);
    if (st != EP_OK)
        return st;
    if ((int)quant < (int)EP_QUANT_BF16 || (int)quant > (int)EP_QUANT_MXFP4_E2M1)
        return EP_ERR_INVALID_ARG;
    const bool quantised = quant != EP_QUANT_BF16;
    const bool mx = quant == EP_QUANT_MXFP8_E4M3 || quant == EP_QUANT_MXFP8_E5M2 ||
                    quant == EP_QUANT_MXFP4_E2M1;
    if (H < 8 || H % 8 != 0 || (quant == EP_QUANT_FP8_E4M3_G128 && H % 128 != 0) ||
        (mx && H % 32 != 0))
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (cap < 0 || (int64_t)E * cap > kI32)
        return EP_ERR_INVALID_ARG;
    if (!ep::ll_dispatch_fits(T, K, H, (int)quant))
        return EP_ERR_UNSUPPORTED;
    const bool rows = (int64_t)E * cap > 0;
    if (!recv_count || !num_dropped || !num_invalid || (T > 0 && (!x || !topk_idx || !slot)) ||
        (rows && T > 0 && !recv_x) || (quantised && rows && T > 0 && !recv_scales))
        return EP_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(recv_x, 16) || (!mx && !aligned(recv_scales, 4)) ||
        !aligned(topk_idx, 4) || !aligned(slot, 4) || !aligned(recv_src, 4) ||
        !aligned(recv_count, 4) || !aligned(num_dropped, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    return hip_status(ep::launch_ll_dispatch(x, T, H, topk_idx, K, E, cap, (int)quant, recv_x,
                                             recv_scales, slot, recv_src, recv_count,
                                             num_dropped, num_invalid,
                                             static_cast<hipStream_t>(stream)));
}

ep_status_t ep_combine(const uint16_t *y, int y_rows, int H, const int32_t *slot,
                       const float *topk_weights, int T, int K, uint16_t *out, void *stream)
{
    if (T < 0 || K < 1 || H < 8 || H % 8 != 0 || (int64_t)T * K > kI32 || y_rows < 0)
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (T > 0 && (!slot || !out || (y_rows > 0 && !y)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(slot, 4) || !aligned(topk_weights, 4))
        return EP_ERR_INVALID_ARG;
    return hip_status(ep::launch_combine(y, y_rows, H, slot, topk_weights, T, K, out,
                                         static_cast<hipStream_t>(stream)));
}

size_t ep_pack_workspace_bytes(int T, int K, int E, int R)
{
    if (check_layout_sizes(T, K, E, R) != EP_OK)
        return 0;
    return ep::make_rank_plan(T, K, E, R).bytes;
}

ep_status_t ep_pack_by_rank(const uint16_t *x, int T, int H, const int32_t *topk_idx,
                            const float *topk_weights, int K, int E, int R, int max_rows,
                            int32_t *tokens_per_rank, int32_t *rank_offsets, uint16_t *send_x,
                            int32_t *send_src, int32_t *send_idx, float *send_w,
                            int32_t *pack_pos, int32_t *num_dropped, void *ws, size_t ws_bytes,
                            void *stream)
{
    ep_status_t st = check_layout_sizes(T, K, E, R);
    if (st != EP_OK)
        return st;
    if (H < 8 || H % 8 != 0 || max_rows < 0)
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (!tokens_per_rank || !rank_offsets || !num_dropped ||
        (T > 0 && (!x || !topk_idx || !pack_pos)) ||
        (T > 0 && max_rows > 0 && (!send_x || !send_src || !send_idx)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(send_x, 16) || !aligned(topk_idx, 4) ||
        !aligned(topk_weights, 4) || !aligned(tokens_per_rank, 4) || !aligned(rank_offsets, 4) ||
        !aligned(send_src, 4) || !aligned(send_idx, 4) || !aligned(send_w, 4) ||
        !aligned(pack_pos, 4) || !aligned(num_dropped, 4))
        return EP_ERR_INVALID_ARG;
    if ((int64_t)T * R > kI32 || (int64_t)max_rows * K > kI32)
        return EP_ERR_INVALID_ARG;
    const ep::RankPlan rp = ep::make_rank_plan(T, K, E, R);
    if ((st = check_ws(ws, ws_bytes, rp.bytes)) != EP_OK)
        return st;
    return hip_status(ep::launch_rank_pack(rp, x, H, topk_idx, topk_weights, E, R, max_rows,
                                           tokens_per_rank, rank_offsets, send_x, send_src,
                                           send_idx, send_w, pack_pos, num_dropped,
                                           static_cast<char *>(ws),
                                           static_cast<hipStream_t>(stream)));
}

ep_status_t ep_combine_partial(const uint16_t *y, int y_rows, int H, const int32_t *slot,
                               const float *weights, int S, int K, float *partial, void *stream)
{
    if (S < 0 || K < 1 || H < 8 || H % 8 != 0 || (int64_t)S * K > kI32 || y_rows < 0)
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (S > 0 && (!slot || !partial || (y_rows > 0 && !y)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(partial, 16) || !aligned(slot, 4) || !aligned(weights, 4))
        return EP_ERR_INVALID_ARG;
    return hip_status(ep::launch_combine_partial(y, y_rows, H, slot, weights, S, K, partial,
                                                 static_cast<hipStream_t>(stream)));
}

ep_status_t ep_combine_ranks(const float *partial, int rows, int H, const int32_t *pack_pos,
                             int T, int R, uint16_t *out, void *stream)
{
    if (T < 0 || R < 1 || rows < 0 || H < 8 || H % 8 != 0 || (int64_t)T * R > kI32)
        return EP_ERR_INVALID_ARG;
    if (R > kMaxRanks || H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (T > 0 && (!pack_pos || !out || (rows > 0 && !partial)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(partial, 16) || !aligned(out, 16) || !aligned(pack_pos, 4))
        return EP_ERR_INVALID_ARG;
    return hip_status(ep::launch_rank_sum(partial, rows, H, pack_pos, T, R, out,
                                          static_cast<hipStream_t>(stream)));
}

ep_status_t ep_dispatch_expert_choice(const uint16_t *x, int T, int H,
                                      const int32_t *token_indices, int E, int C,
                                      uint16_t *recv_x, int32_t *tok_off, int32_t *tok_ent,
                                      int32_t *num_invalid, void *ws, size_t ws_bytes,
                                      void *stream)
{
    if (T < 0 || T >= kI32 || E < 1 || C < 1 || (int64_t)E * C > kI32 || H < 8 || H % 8 != 0)
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (!token_indices || !tok_off || !tok_ent || !num_invalid || !recv_x || (T > 0 && !x))
        return EP_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(recv_x, 16) || !aligned(token_indices, 4) ||
        !aligned(tok_off, 4) || !aligned(tok_ent, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    ep::EcPlan p = ep::make_ec_plan(T, E, C);
    ep_status_t st = check_ws(ws, ws_bytes, p.bytes);
    if (st != EP_OK)
        return st;
    return hip_status(ep::launch_ec_dispatch(p, x, H, token_indices, recv_x, tok_off, tok_ent,
                                             num_invalid, static_cast<char *>(ws),
                                             static_cast<hipStream_t>(stream)));
}

ep_status_t ep_combine_expert_choice(const uint16_t *y, const float *weights, int E, int C, int H,
                                     const int32_t *tok_off, const int32_t *tok_ent, int T,
                                     uint16_t *out, void *stream)
{
    if (T < 0 || T >= kI32 || E < 1 || C < 1 || (int64_t)E * C > kI32 || H < 8 || H % 8 != 0)
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden)
        return EP_ERR_UNSUPPORTED;
    if (T > 0 && (!y || !weights || !tok_off || !tok_ent || !out))
        return EP_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(weights, 4) || !aligned(tok_off, 4) ||
        !aligned(tok_ent, 4))
        return EP_ERR_INVALID_ARG;
    return hip_status(ep::launch_ec_combine(y, weights, E, C, H, tok_off, tok_ent, T, out,
                                            static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- the router
namespace {

ep_status_t check_router_sizes(int T, int E, int K, ep_dtype_t dtype, ep_score_t score)
{
    if (T < 0 || E < 1 || K < 1 || (int64_t)T * K > kI32)
        return EP_ERR_INVALID_ARG;
    if (dtype != EP_DTYPE_BF16 && dtype != EP_DTYPE_F32)
        return EP_ERR_INVALID_ARG;
    if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID)
        return EP_ERR_INVALID_ARG;
    if (E > kMaxExperts)
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

ep_status_t check_sequences(int E, const int32_t *seq_offsets, int S)
{
    if (S < 1 || (!seq_offsets && S != 1) || (int64_t)S * E > kI32)
        return EP_ERR_INVALID_ARG;
    // one block of 512 threads per 16 experts of a sequence: 32-bit grid
    if ((int64_t)S * ((E + 15) / 16) >= 1 << 22)
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

}  // namespace

ep_status_t ep_route(const void *logits, ep_dtype_t dtype, int T, int E, int K, ep_score_t score,
                     const float *bias, int renormalise, float scale, int32_t *topk_idx,
                     float *topk_weights, int32_t *num_invalid, void *stream)
{
    ep_status_t st = check_router_sizes(T, E, K, dtype, score);
    if (st != EP_OK)
        return st;
    if (K > E || (bias && score != EP_SCORE_SIGMOID))
        return EP_ERR_INVALID_ARG;
    if (K > ep::kMaxRouteTopk)
        return EP_ERR_UNSUPPORTED;
    if (T > 0 && (!logits || !topk_idx || !topk_weights))
        return EP_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
        !aligned(topk_weights, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    return hip_status(ep::launch_route(logits, dtype == EP_DTYPE_BF16, T, E, K,
                                       score == EP_SCORE_SIGMOID, bias, renormalise != 0, scale,
                                       topk_idx, topk_weights, num_invalid,
                                       static_cast<hipStream_t>(stream)));
}

size_t ep_balance_workspace_bytes(int T, int E, int S)
{
    if (check_router_sizes(T, E, 1, EP_DTYPE_F32, EP_SCORE_SOFTMAX) != EP_OK || S < 1 ||
        (int64_t)S * E > kI32)
        return 0;
    return ep::make_balance_plan(T, E, S).bytes;
}

ep_status_t ep_balance_loss(const void *logits, ep_dtype_t dtype, int T, int E,
                            const int32_t *topk_idx, int K, ep_score_t score,
                            const int32_t *seq_offsets, int S, float coef, int32_t *counts,
                            float *slope, float *loss, int32_t *num_invalid, void *ws,
                            size_t ws_bytes, void *stream)
{
    ep_status_t st = check_router_sizes(T, E, K, dtype, score);
    if (st == EP_OK)
        st = check_sequences(E, seq_offsets, S);
    if (st != EP_OK)
        return st;
    if ((T > 0 && (!logits || !topk_idx)) || !counts || !slope || !loss || !num_invalid)
        return EP_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(topk_idx, 4) || !aligned(seq_offsets, 4) ||
        !aligned(counts, 4) || !aligned(slope, 4) || !aligned(loss, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    const ep::BalancePlan p = ep::make_balance_plan(T, E, S);
    if ((st = check_ws(ws, ws_bytes, p.bytes)) != EP_OK)
        return st;
    return hip_status(ep::launch_balance(p, logits, dtype == EP_DTYPE_BF16, topk_idx, K,
                                         score == EP_SCORE_SIGMOID, seq_offsets, coef, counts,
                                         slope, loss, num_invalid, static_cast<char *>(ws),
                                         static_cast<hipStream_t>(stream)));
}

ep_status_t ep_router_backward(const void *logits, ep_dtype_t dtype, int T, int E, int K,
                               ep_score_t score, int renormalise, float scale,
                               const int32_t *topk_idx, const float *d_weights, const float *slope,
                               const int32_t *seq_offsets, int S, const float *d_loss,
                               void *d_logits, void *stream)
{
    ep_status_t st = check_router_sizes(T, E, K, dtype, score);
    if (st == EP_OK && slope)
        st = check_sequences(E, seq_offsets, S);
    if (st != EP_OK)
        return st;
    if (T > 0 && !d_weights && !slope)
        return EP_ERR_INVALID_ARG;
    if (d_weights && K > ep::kMaxRouteTopk)
        return EP_ERR_UNSUPPORTED;
    if ((slope && !d_loss) || (T > 0 && (!logits || !d_logits || (d_weights && !topk_idx))))
        return EP_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(d_logits, 16) || !aligned(topk_idx, 4) ||
        !aligned(d_weights, 4) || !aligned(slope, 4) || !aligned(seq_offsets, 4) ||
        !aligned(d_loss, 4))
        return EP_ERR_INVALID_ARG;
    return hip_status(ep::launch_router_backward(
        logits, dtype == EP_DTYPE_BF16, T, E, K, score == EP_SCORE_SIGMOID, renormalise != 0,
        scale, topk_idx, d_weights, slope, seq_offsets, S, d_loss, d_logits,
        static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- adapters
namespace {

ep_status_t check_adapter_sizes(int T, int H, int O, int E, int K, int r)
{
    if (T < 0 || K < 1 || E < 1 || H < 8 || H % 8 != 0 || O < 8 || O % 8 != 0 || r < 8 ||
        r % 8 != 0 || (int64_t)T * K > kI32)
        return EP_ERR_INVALID_ARG;
    if (E > kMaxExperts || H > ep::kMaxAdapterWidth || O > ep::kMaxAdapterWidth || r > ep::kMaxAdapterRank ||
        K > ep::kMaxAdapterTopk)
        return EP_ERR_UNSUPPORTED;
    // tiles of 128 tokens (larger calls) times blocks of 128 channels, 256 threads each: 32-bit grids
    const int64_t tiles = ((int64_t)T + 127) / 128, blocks = ((H > O ? H : O) + 127) / 128;
    if (tiles * (blocks > 16 ? blocks : 16) >= 1 << 23 || blocks * E >= 1 << 22)
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

// The operands of both directions.
ep_status_t check_adapter_args(const uint16_t *x, int T, const uint16_t *weight, const uint16_t *a,
                               const uint16_t *b, const int32_t *topk_idx,
                               const float *topk_weights, const void *state)
{
    if (!weight || !a || !b || (T > 0 && (!x || !topk_idx)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(a, 16) || !aligned(b, 16) ||
        !aligned(topk_idx, 4) || !aligned(topk_weights, 4) || !aligned(state, 256))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

}  // namespace

size_t ep_adapter_state_bytes(int T, int H, int O, int E, int K, int r)
{
    if (check_adapter_sizes(T, H, O, E, K, r) != EP_OK)
        return 0;
    return ep::make_adapter_plan(T, H, O, E, K, r).state_bytes;
}

size_t ep_adapter_workspace_bytes(int T, int H, int O, int E, int K, int r, int backward)
{
    if (check_adapter_sizes(T, H, O, E, K, r) != EP_OK)
        return 0;
    const ep::AdapterPlan p = ep::make_adapter_plan(T, H, O, E, K, r);
    return backward ? p.back_bytes : p.ws_bytes;
}

ep_status_t ep_adapter_project(const uint16_t *x, int T, int H, const uint16_t *weight, int O,
                               const uint16_t *a, const uint16_t *b, int E, int r,
                               const int32_t *topk_idx, const float *topk_weights, int K,
                               float scale, uint16_t *out, int32_t *num_invalid, void *state,
                               size_t state_bytes, void *ws, size_t ws_bytes, void *stream)
{
    ep_status_t st = check_adapter_sizes(T, H, O, E, K, r);
    if (st == EP_OK)
        st = check_adapter_args(x, T, weight, a, b, topk_idx, topk_weights, state);
    if (st != EP_OK)
        return st;
    if ((T > 0 && !out) || !aligned(out, 16) || !num_invalid || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    const ep::AdapterPlan p = ep::make_adapter_plan(T, H, O, E, K, r);
    if ((st = check_ws(state, state_bytes, p.state_bytes)) != EP_OK ||
        (st = check_ws(ws, ws_bytes, p.ws_bytes)) != EP_OK)
        return st;
    return hip_status(ep::launch_adapter(p, x, weight, a, b, topk_idx, topk_weights, scale, out,
                                         num_invalid, static_cast<char *>(state),
                                         static_cast<char *>(ws),
                                         static_cast<hipStream_t>(stream)));
}

ep_status_t ep_adapter_project_backward(const uint16_t *d_out, const uint16_t *x, int T, int H,
                                        const uint16_t *weight, int O, const uint16_t *a,
                                        const uint16_t *b, int E, int r, const int32_t *topk_idx,
                                        const float *topk_weights, int K, float scale,
                                        const void *state, size_t state_bytes, uint16_t *dx,
                                        uint16_t *da, uint16_t *db, float *d_weights, void *ws,
                                        size_t ws_bytes, void *stream)
{
    ep_status_t st = check_adapter_sizes(T, H, O, E, K, r);
    if (st == EP_OK)
        st = check_adapter_args(x, T, weight, a, b, topk_idx, topk_weights, state);
    if (st != EP_OK)
        return st;
    if ((T > 0 && (!d_out || (!dx && !da && !db && !d_weights))) || !aligned(d_out, 16) ||
        !aligned(dx, 16) || !aligned(da, 16) || !aligned(db, 16) || !aligned(d_weights, 4))
        return EP_ERR_INVALID_ARG;
    const ep::AdapterPlan p = ep::make_adapter_plan(T, H, O, E, K, r);
    if ((st = check_ws(state, state_bytes, p.state_bytes)) != EP_OK ||
        (st = check_ws(ws, ws_bytes, p.back_bytes)) != EP_OK)
        return st;
    return hip_status(ep::launch_adapter_backward(
        p, d_out, x, weight, a, b, topk_idx, topk_weights, scale,
        static_cast<char *>(const_cast<void *>(state)), dx, da, db, d_weights,
        static_cast<char *>(ws), static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- microscaled tensors
namespace {

bool is_mx(ep_quant_t quant)
{
    return quant == EP_QUANT_MXFP8_E4M3 || quant == EP_QUANT_MXFP8_E5M2 || quant == EP_QUANT_MXFP4_E2M1;
}

ep_status_t check_mx(const void *bf16, int rows, int H, ep_quant_t quant, const void *codes, const uint8_t *scales)
{
    if (rows < 0 || H < 32 || H % 32 != 0 || !is_mx(quant))
        return EP_ERR_INVALID_ARG;
    if (H > kMaxHidden || (int64_t)rows * (H / 8) > (int64_t)1 << 33)
        return EP_ERR_UNSUPPORTED;
    if (rows > 0 && (!bf16 || !codes || !scales))
        return EP_ERR_INVALID_ARG;
    if (!aligned(bf16, 16) || !aligned(codes, 16))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

}  // namespace

ep_status_t ep_mx_quantize(const uint16_t *x, int rows, int H, ep_quant_t quant, void *codes, uint8_t *scales,
                           void *stream)
{
    const ep_status_t st = check_mx(x, rows, H, quant, codes, scales);
    if (st != EP_OK)
        return st;
    return hip_status(ep::launch_mx_quantize(x, rows, H, quant, codes, scales, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_mx_dequantize(const void *codes, const uint8_t *scales, int rows, int H, ep_quant_t quant,
                             uint16_t *out, void *stream)
{
    const ep_status_t st = check_mx(out, rows, H, quant, codes, scales);
    if (st != EP_OK)
        return st;
    return hip_status(ep::launch_mx_dequantize(codes, scales, rows, H, quant, out, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- the experts' products
namespace {

// The rows, the weight, and the sizes of both directions.
ep_status_t check_expert(const void *x, const uint8_t *x_scales, ep_quant_t x_quant, int rows, const uint8_t *weight,
                         const uint8_t *weight_scales, int E, int O, int H, const int32_t *offsets,
                         const int32_t *counts, int cap, ep_activation_t activation)
{
    if (rows < 0 || E < 1 || H < 32 || H % 32 != 0 || O < 8 || (x_quant != EP_QUANT_BF16 && !is_mx(x_quant)) ||
        (activation != EP_ACT_NONE && activation != EP_ACT_SWIGLU))
        return EP_ERR_INVALID_ARG;
    if (O % (activation == EP_ACT_SWIGLU ? 16 : 8) != 0)
        return EP_ERR_INVALID_ARG;
    // rows by offsets, or E * cap of them
    if (offsets ? (counts || cap != 0) : (cap < 0 || (int64_t)E * cap != rows))
        return EP_ERR_INVALID_ARG;
    if (E > kMaxExperts || H > ep::kMaxAdapterWidth || O > ep::kMaxAdapterWidth || (int64_t)O * H >= (int64_t)1 << 31)
        return EP_ERR_UNSUPPORTED;
    // tiles of 32 rows and more by 64 columns and more, 256 threads each: 32-bit grids
    const int64_t tiles = ((int64_t)rows + 31) / 32 + E, blocks = ((H > O ? H : O) + 63) / 64;
    if (tiles * blocks >= 1 << 23)
        return EP_ERR_UNSUPPORTED;
    if (!weight || !weight_scales || (rows > 0 && (!x || (x_quant != EP_QUANT_BF16 && !x_scales))))
        return EP_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(offsets, 4) || !aligned(counts, 4))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

}  // namespace

ep_status_t ep_expert_product(const void *x, const uint8_t *x_scales, ep_quant_t x_quant, int rows,
                              const uint8_t *weight, const uint8_t *weight_scales, int E, int O, int H,
                              const int32_t *offsets, const int32_t *counts, int cap, ep_activation_t activation,
                              ep_quant_t y_quant, void *y, uint8_t *y_scales, void *stream)
{
    const ep_status_t st = check_expert(x, x_scales, x_quant, rows, weight, weight_scales, E, O, H, offsets, counts,
                                        cap, activation);
    if (st != EP_OK)
        return st;
    const bool gated = activation == EP_ACT_SWIGLU;
    const int width = gated ? O / 2 : O;
    const bool coded = y_quant != EP_QUANT_BF16;
    if ((coded && !is_mx(y_quant)) || (coded && width % 32 != 0) || (rows > 0 && (!y || (coded && !y_scales))) ||
        !aligned(y, 16))
        return EP_ERR_INVALID_ARG;
    if (rows == 0)
        return EP_OK;
    const ep::ExpertRows m{offsets, counts, rows, cap, E};
    const ep::ExpertIn in{x, x_scales, weight, weight_scales, O, H, gated ? O / 2 : 0};
    const ep::ExpertOut out{y, y_scales, nullptr, width, gated ? ep::kExpertGated : ep::kExpertPlain, y_quant};
    return hip_status(ep::launch_expert(m, in, out, x_quant, static_cast<hipStream_t>(stream)));
}

size_t ep_expert_workspace_bytes(int rows, int O, ep_activation_t activation)
{
    if (rows < 0 || O < 8 || (activation != EP_ACT_NONE && activation != EP_ACT_SWIGLU))
        return 0;
    return activation == EP_ACT_SWIGLU && rows > 0 ? ep::align256((size_t)rows * O * 2) : 256;
}

ep_status_t ep_expert_product_backward(const uint16_t *d_y, const void *x, const uint8_t *x_scales,
                                       ep_quant_t x_quant, int rows, const uint8_t *weight,
                                       const uint8_t *weight_scales, int E, int O, int H, const int32_t *offsets,
                                       const int32_t *counts, int cap, ep_activation_t activation, uint16_t *dx,
                                       void *ws, size_t ws_bytes, void *stream)
{
    // without an activation the rows themselves are not read
    const bool gated = activation == EP_ACT_SWIGLU;
    ep_status_t st = check_expert(gated ? x : d_y, gated ? x_scales : nullptr, gated ? x_quant : EP_QUANT_BF16, rows,
                                  weight, weight_scales, E, O, H, offsets, counts, cap, activation);
    if (st != EP_OK)
        return st;
    if ((rows > 0 && (!d_y || !dx)) || !aligned(d_y, 16) || !aligned(dx, 16))
        return EP_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, ep_expert_workspace_bytes(rows, O, activation))) != EP_OK)
        return st;
    if (rows == 0)
        return EP_OK;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const ep::ExpertRows m{offsets, counts, rows, cap, E};
    const void *d = d_y;
    if (gated) {
        const ep::ExpertIn in{x, x_scales, weight, weight_scales, O, H, O / 2};
        const ep::ExpertOut out{ws, nullptr, d_y, O / 2, ep::kExpertGrad, EP_QUANT_BF16};
        if ((st = hip_status(ep::launch_expert(m, in, out, x_quant, s))) != EP_OK)
            return st;
        d = ws;
    }
    const ep::ExpertIn in{d, nullptr, weight, weight_scales, O, H, 0};
    const ep::ExpertOut out{dx, nullptr, nullptr, H, ep::kExpertPlain, EP_QUANT_BF16};
    return hip_status(ep::launch_expert_across(m, in, out, s));
}

// ---------------------------------------------------------------- a few tokens' layer
namespace {

ep_status_t check_few_sizes(int T, int K, int E, int H, int I)
{
    if (T < 0 || K < 1 || E < 1 || H < 8 || H % 8 != 0 || I < 8 || I % 8 != 0)
        return EP_ERR_INVALID_ARG;
    if (T > ep::kFewTokens || (int64_t)T * K > ep::kLlMaxEntries || K > ep::kLlMaxTopk || E > kMaxExperts ||
        H > ep::kMaxAdapterWidth || I > ep::kMaxAdapterWidth)
        return EP_ERR_UNSUPPORTED;
    const int64_t most = (int64_t)T * K < E ? (int64_t)T * K : E;
    if (most * ((H > I ? H : I) / 16 + 1) >= 1 << 22)       // blocks of up to 512 threads: 32-bit grids
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

}  // namespace

size_t ep_low_latency_experts_workspace_bytes(int T, int K, int E, int H, int I)
{
    return check_few_sizes(T, K, E, H, I) == EP_OK ? ep::make_few_plan(T, K, E, H, I, false).bytes : 0;
}

ep_status_t ep_low_latency_experts(const uint16_t *x, int T, int H, const int32_t *topk_idx,
                                   const float *topk_weights, int K, const void *up, const uint8_t *up_scales,
                                   const void *down, const uint8_t *down_scales, int E, int I, uint16_t *out,
                                   int32_t *num_invalid, void *ws, size_t ws_bytes, void *stream)
{
    ep_status_t st = check_few_sizes(T, K, E, H, I);
    if (st != EP_OK)
        return st;
    const bool coded = up_scales || down_scales;
    if (coded && (!up_scales || !down_scales || H % 32 != 0 || I % 32 != 0))
        return EP_ERR_INVALID_ARG;
    if (!up || !down || !num_invalid || (T > 0 && (!x || !topk_idx || !out)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(up, 16) || !aligned(down, 16) || !aligned(out, 16) || !aligned(topk_idx, 4) ||
        !aligned(topk_weights, 4) || !aligned(num_invalid, 4))
        return EP_ERR_INVALID_ARG;
    const ep::FewPlan p = ep::make_few_plan(T, K, E, H, I, coded);
    if ((st = check_ws(ws, ws_bytes, p.bytes)) != EP_OK)
        return st;
    return hip_status(ep::launch_few(p, x, topk_idx, topk_weights, up, up_scales, down, down_scales, out, num_invalid,
                                     static_cast<char *>(ws), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
