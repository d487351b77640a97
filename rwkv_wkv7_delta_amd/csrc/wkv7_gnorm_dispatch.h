// wkv7_gnorm_dispatch.h -- from a launch plan to run<T, V, P, K, gate, silu> (the
// variants that the plan chooses from), for the body of a launcher.
#pragma once

#define WKV7_GN_MODE(T, V, P, K, gate) \
    return p.silu ? run<T, V, P, K, gate, true>(p, stream) : run<T, V, P, K, gate, false>(p, stream);
#define WKV7_GN(T, V, P, K)                                                                    \
    if (p.plan.vec == V && p.plan.lanes == P && p.plan.each == K) {                            \
        if (p.gate == 0) WKV7_GN_MODE(T, V, P, K, 0)                                           \
        if (p.gate == 1) WKV7_GN_MODE(T, V, P, K, 1)                                           \
        WKV7_GN_MODE(T, V, P, K, 2)                                                            \
    }
#define WKV7_GN_ALL(T, V)                                                                      \
    WKV7_GN(T, V, 4, 1) WKV7_GN(T, V, 8, 1) WKV7_GN(T, V, 16, 1) WKV7_GN(T, V, 32, 1)          \
    WKV7_GN(T, V, 64, 1) WKV7_GN(T, V, 64, 2) WKV7_GN(T, V, 128, 2) WKV7_GN(T, V, 256, 2)      \
    WKV7_GN(T, V, 512, 2) WKV7_GN(T, V, 256, 0)
#define WKV7_GN_BF16 WKV7_GN_ALL(bf16_t, 8) WKV7_GN_ALL(bf16_t, 2) WKV7_GN_ALL(bf16_t, 1)
#define WKV7_GN_F32 WKV7_GN_ALL(float, 4) WKV7_GN_ALL(float, 1)
