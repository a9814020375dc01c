// ep_mx.hip -- bf16 tensors to microscaled codes and back.
//
// A block of 32 channels has the scale 2^E, E = floor(log2 max|x|) - emax (2 for
// e2m1, 8 and 15 for the 8-bit formats), and the codes RNE(x 2^-E), saturating:
// the bytes that the dispatch's MX modes make of the same rows.  As a row is
// whole blocks, the tensor is one run of them whatever its shape.
//
// Bound by memory: 2 bytes in and 17/32 (or 33/32) out for a channel.  A lane
// takes 8 channels (16 bytes), four lanes a block; the maximum goes round by
// quad permutations.  470 M values (16 matrices of 4096 x 7168) to MXFP4 in 178 us
// and back in 166 (6.7 and 7.2 TB/s); 128 rows of 7168 to MXFP8 in 3.1 and back in
// 2.9, the launch's own time.
#include "ep_common.h"
#include "ep_internal.h"

namespace ep {

namespace {

constexpr int kMxThreads = 256;
constexpr int kMxSteps = 4;         // loads of 16 bytes in flight per lane

// The larger of the quad's four values.
__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, dpp_f<0xB1, 0xF>(0.0f, v));        // lanes 1, 0, 3, 2
    return fmaxf(v, dpp_f<0x4E, 0xF>(0.0f, v));     // lanes 2, 3, 0, 1
}

template <int MODE>
__global__ void __launch_bounds__(kMxThreads)
mx_quantize_kernel(const uint16_t *__restrict__ x, int64_t pieces, uint8_t *__restrict__ codes,
                   uint8_t *__restrict__ scales)
{
    const int64_t first = (int64_t)blockIdx.x * (kMxThreads * kMxSteps) + threadIdx.x;
    u32x4 in[kMxSteps];
#pragma unroll
    for (int s = 0; s < kMxSteps; ++s) {
        const int64_t p = first + s * kMxThreads;
        in[s] = p < pieces ? ld16_nt(x + p * 8) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int s = 0; s < kMxSteps; ++s) {
        const int64_t p = first + s * kMxThreads;       // pieces % 4 == 0: whole quads
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(in[s][i]);
            v[2 * i + 1] = bf16_hi(in[s][i]);
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = fmaxf(top, fabsf(v[i]));
        const uint32_t code = mx_scale_code<MODE>(quad_max(top));
        if (p >= pieces)
            continue;
        if constexpr (MODE == kQuantMxE2M1) {
            *reinterpret_cast<uint32_t *>(codes + p * 4) = e2m1x8_scaled(v, code);
        } else {
            const u32x2 w = {mx8x4<MODE>(v[0], v[1], v[2], v[3], code), mx8x4<MODE>(v[4], v[5], v[6], v[7], code)};
            *reinterpret_cast<u32x2 *>(codes + p * 8) = w;
        }
        if (p % 4 == 0)
            scales[p / 4] = (uint8_t)code;
    }
}

// Back: code * 2^E, rounded to bf16 (which changes only values below 2^-126).
template <int MODE>
__global__ void __launch_bounds__(kMxThreads)
mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t pieces,
                     uint16_t *__restrict__ out)
{
    const int64_t first = (int64_t)blockIdx.x * (kMxThreads * kMxSteps) + threadIdx.x;
    u32x2 in[kMxSteps];
    uint32_t sc[kMxSteps];
#pragma unroll
    for (int s = 0; s < kMxSteps; ++s) {
        const int64_t p = first + s * kMxThreads;
        in[s] = u32x2{0u, 0u};
        sc[s] = 127u;
        if (p < pieces) {
            if constexpr (MODE == kQuantMxE2M1)
                in[s][0] = *reinterpret_cast<const uint32_t *>(codes + p * 4);
            else
                in[s] = *reinterpret_cast<const u32x2 *>(codes + p * 8);
            sc[s] = scales[p / 4];
        }
    }
#pragma unroll
    for (int s = 0; s < kMxSteps; ++s) {
        const int64_t p = first + s * kMxThreads;
        if (p < pieces)
            st16_nt(out + p * 8, MODE == kQuantMxE2M1 ? e2m1_bf16x8(in[s][0], sc[s]) : mx8_bf16x8<MODE>(in[s], sc[s]));
    }
}

unsigned mx_blocks(int64_t pieces)
{
    const int64_t per = kMxThreads * kMxSteps;
    return (unsigned)((pieces + per - 1) / per);
}

}  // namespace

hipError_t launch_mx_quantize(const uint16_t *x, int64_t rows, int H, int mode, void *codes, uint8_t *scales,
                              hipStream_t s)
{
    const int64_t pieces = rows * (H / 8);
    if (pieces == 0)
        return hipSuccess;
    uint8_t *c = static_cast<uint8_t *>(codes);
    switch (mode) {
        case kQuantMxE4M3: mx_quantize_kernel<kQuantMxE4M3><<<mx_blocks(pieces), kMxThreads, 0, s>>>(x, pieces, c, scales); break;
        case kQuantMxE5M2: mx_quantize_kernel<kQuantMxE5M2><<<mx_blocks(pieces), kMxThreads, 0, s>>>(x, pieces, c, scales); break;
        default: mx_quantize_kernel<kQuantMxE2M1><<<mx_blocks(pieces), kMxThreads, 0, s>>>(x, pieces, c, scales); break;
    }
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void *codes, const uint8_t *scales, int64_t rows, int H, int mode,
                                uint16_t *out, hipStream_t s)
{
    const int64_t pieces = rows * (H / 8);
    if (pieces == 0)
        return hipSuccess;
    const uint8_t *c = static_cast<const uint8_t *>(codes);
    switch (mode) {
        case kQuantMxE4M3: mx_dequantize_kernel<kQuantMxE4M3><<<mx_blocks(pieces), kMxThreads, 0, s>>>(c, scales, pieces, out); break;
        case kQuantMxE5M2: mx_dequantize_kernel<kQuantMxE5M2><<<mx_blocks(pieces), kMxThreads, 0, s>>>(c, scales, pieces, out); break;
        default: mx_dequantize_kernel<kQuantMxE2M1><<<mx_blocks(pieces), kMxThreads, 0, s>>>(c, scales, pieces, out); break;
    }
    return hipGetLastError();
}

}  // namespace ep
