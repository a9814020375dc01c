// Host-side paths of the experts' C entry points that run without a GPU: the
// sizes over a wide grid and at the largest arguments that they accept, and
// argument checks there, which return before anything is enqueued.  Built with
// the host pass under AddressSanitizer and UndefinedBehaviorSanitizer, so that
// an overflow in the size arithmetic is reported.  Exit status 0 = clean.
// Test infrastructure: built and run by tests/test_experts_sanitize.py.
#include <stdint.h>
#include <stdio.h>

#include "ep.h"

#include <hip/hip_runtime.h>

#include "ep_internal.h"

static int failures = 0;

static void expect(bool ok, const char *what, long long a, long long b)
{
    if (!ok) {
        fprintf(stderr, "%s (%lld, %lld)\n", what, a, b);
        ++failures;
    }
}

int main()
{
    const int kMost = 2147483647;
    const int Ts[] = {0, 1, 2, 63, 64, 65, 127, 128}, Ks[] = {1, 2, 8, 31, 32, 64}, Es[] = {1, 2, 8, 257, 4096};
    const int Ws[] = {8, 32, 72, 4096, 7168, 65536, 1 << 20};
    for (int T : Ts)
        for (int K : Ks)
            for (int E : Es)
                for (int H : Ws)
                    for (int I : Ws) {
                        const size_t b = ep_low_latency_experts_workspace_bytes(T, K, E, H, I);
                        const long long most = (long long)T * K < E ? (long long)T * K : E;
                        const bool fits = T * K <= 4096 && most * ((H > I ? H : I) / 16 + 1) < 1 << 22;
                        expect((b > 0) == fits, "few: accepted", T * K, H);
                        if (!fits)
                            continue;
                        // h in two parts, the entries' outputs, the tables; the same for either type of weights
                        const size_t n = (size_t)T * K;
                        expect(b % 256 == 0 && b >= n * I * 4 + n * H * 4, "few: workspace", T, H);
                        for (int fp4 = 0; fp4 < 2; ++fp4) {
                            const ep::FewPlan p = ep::make_few_plan(T, K, E, H, I, fp4 != 0);
                            expect(p.bytes == b, "few: one size", T, H);
                            // every slice has its counter, every buffer of shared columns is in reach
                            expect(p.off_arrived + (size_t)p.slices * 4 <= p.off_named, "few: counters", p.slices, H);
                            expect(!p.wide || ((long long)T * H * 2 <= kMost && p.lower * 4 <= kMost), "few: reach", T, I);
                            expect(p.stage_bytes >= 0 && p.stage_bytes <= 32 << 10, "few: LDS", T, H);
                            // 32-bit grids: tokens in lots of 32 at least
                            const long long blocks = most * (p.wide ? 4 : 1) * (p.slices > p.slices_up ? p.slices : p.slices_up);
                            expect(blocks * 256 <= kMost, "few: grid", blocks, H);
                        }
                        // a buffer too small, or none, is refused before a launch
                        int x[4] = {0, 0, 0, 0};
                        const uint16_t *in = reinterpret_cast<const uint16_t *>(((uintptr_t)x + 15) & ~(uintptr_t)15);
                        expect(ep_low_latency_experts(in, T, H, x, nullptr, K, in, nullptr, in, nullptr, E, I,
                                                      const_cast<uint16_t *>(in), x, nullptr, b, nullptr) != EP_OK,
                               "few: no workspace", T, H);
                    }
    expect(ep_low_latency_experts_workspace_bytes(129, 1, 1, 8, 8) == 0, "few: T", 129, 0);
    expect(ep_low_latency_experts_workspace_bytes(kMost, kMost, 1, 8, 8) == 0, "few: T, K", kMost, 0);
    expect(ep_low_latency_experts_workspace_bytes(1, 1, kMost, 8, 8) == 0, "few: E", kMost, 0);
    expect(ep_low_latency_experts_workspace_bytes(1, 1, 1, kMost - 7, 8) == 0, "few: H", kMost, 0);

    // the products: at the largest sizes every call is refused for its missing operands or for its sizes
    const int rows[] = {0, 1, 255, 1 << 20, 1 << 27, kMost - 31, kMost}, Os[] = {8, 16, 4096, 1 << 20, kMost - 7};
    const int Hs[] = {32, 4096, 1 << 20, kMost - 31}, quants[] = {EP_QUANT_BF16, EP_QUANT_MXFP8_E4M3, EP_QUANT_MXFP4_E2M1};
    for (int r : rows)
        for (int O : Os) {
            for (int act = EP_ACT_NONE; act <= EP_ACT_SWIGLU; ++act) {
                const size_t b = ep_expert_workspace_bytes(r, O, act);
                expect(b >= 256 && (act == EP_ACT_NONE || b >= (size_t)r * O * 2), "products: workspace", r, O);
                for (int H : Hs)
                    for (int E : Es)
                        for (int q : quants) {
                            int32_t off[2] = {0, 0};
                            expect(ep_expert_product(nullptr, nullptr, q, r, nullptr, nullptr, E, O, H, off, nullptr, 0,
                                                     act, EP_QUANT_BF16, nullptr, nullptr, nullptr) != EP_OK,
                                   "products: no operands", r, O);
                            expect(ep_expert_product(nullptr, nullptr, q, r, nullptr, nullptr, E, O, H, nullptr, nullptr,
                                                     r / E, act, EP_QUANT_BF16, nullptr, nullptr, nullptr) != EP_OK,
                                   "products: padded, no operands", r, O);
                        }
            }
            for (int q : quants)
                expect(ep_mx_quantize(nullptr, r, O, q, nullptr, nullptr, nullptr) != EP_OK || r == 0, "quantise: no operands",
                       r, O);
        }
    expect(ep_expert_workspace_bytes(-1, 8, EP_ACT_NONE) == 0, "products: rows < 0", -1, 0);
    expect(ep_expert_workspace_bytes(1, 8, 2) == 0, "products: activation", 2, 0);
    if (failures == 0)
        printf("run clean\n");
    return failures ? 1 : 0;
}
