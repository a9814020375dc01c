// Host-side paths of the router's and the adapters' C entry points that run
// without a GPU: the sizes over a wide grid and at the largest arguments that
// they accept, and argument checks there, which return before anything is
// enqueued.  Built with the host pass under AddressSanitizer and
// UndefinedBehaviorSanitizer, so that an overflow in the size arithmetic is
// reported.  Exit status 0 = clean.  With arguments "T,H,O,E,K,r" it prints the
// form of the adapters' projection that each takes instead.
// Test infrastructure: built and run by tests/test_operators_sanitize.py.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

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

// Tokens of a tile, columns of the forward's tiles and of those of dx.
static int print_form(const char *arg)
{
    int T, H, O, E, K, r;
    if (sscanf(arg, "%d,%d,%d,%d,%d,%d", &T, &H, &O, &E, &K, &r) != 6)
        return 1;
    const ep::AdapterPlan p = ep::make_adapter_plan(T, H, O, E, K, r);
    printf("%d,%d,%d\n", p.BM, ep::adapter_tile_columns(p, O, false), ep::adapter_tile_columns(p, H, true));
    return 0;
}

int main(int argc, char **argv)
{
    for (int i = 1; i < argc; ++i)
        if (print_form(argv[i]))
            return 1;
    if (argc > 1)
        return 0;
    const long long kMost = 2147483647LL;
    const long long Ts[] = {0, 1, 15, 16, 17, 128, 129, 4095, 4096, 4097, 300000, 1 << 20, 1 << 28, 1LL << 30,
                            kMost - 8388607, kMost - 400, kMost - 1, kMost};
    const int Es[] = {1, 2, 8, 37, 256, 384, 1000, 4096};
    const int Ss[] = {1, 2, 7, 1000, 16383};
    // the balance loss: at most 256 chunks and a partial row for each of them and of the sequences
    for (long long T : Ts)
        for (int E : Es)
            for (int S : Ss) {
                if ((long long)S * E > kMost)
                    continue;
                const size_t b = ep_balance_workspace_bytes((int)T, E, S);
                const size_t most = (256 + (size_t)S) * (2 * (size_t)E + 4) * 4 + (size_t)S * ((E + 15) / 16) * 8 +
                                    (size_t)S * 12 + 5 * 256;
                expect(b > 0 && b % 256 == 0 && b <= most, "balance workspace", T, E);
            }
    expect(ep_balance_workspace_bytes(-1, 8, 1) == 0, "balance: T < 0", -1, 0);
    expect(ep_balance_workspace_bytes(4, 4097, 1) == 0, "balance: E", 4097, 0);
    expect(ep_balance_workspace_bytes(4, 8, 0) == 0, "balance: S", 0, 0);
    // the adapters: every accepted size has a state and workspaces
    const int Ws[] = {8, 72, 4096, 7168, 1 << 20}, Ks[] = {1, 2, 8, 64}, rs[] = {8, 24, 128};
    for (long long T : Ts)
        for (int H : Ws)
            for (int O : Ws)
                for (int E : Es)
                    for (int K : Ks)
                        for (int r : rs) {
                            const size_t s = ep_adapter_state_bytes((int)T, H, O, E, K, r);
                            const size_t f = ep_adapter_workspace_bytes((int)T, H, O, E, K, r, 0);
                            const size_t b = ep_adapter_workspace_bytes((int)T, H, O, E, K, r, 1);
                            expect((s == 0) == (f == 0) && (s == 0) == (b == 0), "adapters: all or none", T, H);
                            if (s == 0)
                                continue;
                            const size_t entries = (size_t)T * K * r * 4;
                            expect(s % 256 == 0 && f % 256 == 0 && b % 256 == 0, "adapters: whole 256 bytes", T, H);
                            expect(f >= entries && b >= 2 * entries, "adapters: room for every entry", T, K);
                            expect(T <= 128 || s >= entries, "adapters: the state's sums", T, K);
                        }
    expect(ep_adapter_state_bytes((int)kMost, 8, 8, 1, 1, 8) == 0, "adapters: T beyond the grid", kMost, 0);
    // checks at the largest arguments, each refused for one other argument
    int32_t i4[64] = {0};
    uint16_t h2[64] = {0};
    float f4[64] = {0};
    alignas(256) static char ws[1 << 12];
    const ep_status_t inval = EP_ERR_INVALID_ARG, unsup = EP_ERR_UNSUPPORTED;
    expect(ep_route(nullptr, EP_DTYPE_F32, (int)kMost, 4096, 1, EP_SCORE_SOFTMAX, nullptr, 1, 1.0f, i4, f4, i4,
                    nullptr) == inval, "route: null logits", 0, 0);
    expect(ep_route(nullptr, EP_DTYPE_F32, (int)kMost, 4096, 2, EP_SCORE_SOFTMAX, nullptr, 1, 1.0f, i4, f4, i4,
                    nullptr) == inval, "route: T*K beyond 2^31", kMost, 2);
    expect(ep_balance_loss(f4, EP_DTYPE_F32, (int)kMost, 4096, i4, 1, EP_SCORE_SOFTMAX, i4, 1 << 20, 1.0f, i4, f4,
                           f4, i4, ws, sizeof ws, nullptr) == inval, "balance: S*E beyond 2^31", 1 << 20, 4096);
    alignas(16) static float f16[64];
    expect(ep_balance_loss(f16, EP_DTYPE_F32, (int)kMost, 1, i4, 1, EP_SCORE_SOFTMAX, i4, 1 << 22, 1.0f, i4, f4,
                           f4, i4, ws, sizeof ws, nullptr) == unsup, "balance: grid", 1 << 22, 1);
    expect(ep_balance_loss(f16, EP_DTYPE_F32, (int)kMost, 4096, i4, 1, EP_SCORE_SOFTMAX, nullptr, 1, 1.0f, i4, f4,
                           f4, i4, ws, sizeof ws, nullptr) == EP_ERR_WORKSPACE, "balance: workspace", 0, 0);
    expect(ep_router_backward(f16, EP_DTYPE_F32, (int)kMost, 4096, 1, EP_SCORE_SOFTMAX, 1, 1.0f, i4, nullptr,
                              nullptr, nullptr, 1, nullptr, f16, nullptr) == inval, "backward: nothing to do", 0, 0);
    expect(ep_adapter_project(h2, 1 << 26, 8, h2, 8, h2, h2, 1, 8, i4, nullptr, 1, 1.0f, h2, i4, ws, sizeof ws, ws,
                              sizeof ws, nullptr) == unsup, "adapters: grid", 1 << 26, 8);
    if (failures) {
        fprintf(stderr, "%d check(s) failed\n", failures);
        return 1;
    }
    printf("operators host sanitize run clean\n");
    return 0;
}
