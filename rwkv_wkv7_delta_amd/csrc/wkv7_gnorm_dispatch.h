// wkv7_gnorm_dispatch.h -- the body of a launcher: run<T, V, P, K> of the plan
// (the variants that plan_gnorm chooses from).
#define WKV7_GN(T, V, P, K) \
    if (p.plan.vec == V && p.plan.lanes == P && p.plan.each == K) return run<T, V, P, K>(p, stream);
#define WKV7_GN_ALL(T, V)                                                                      \
    WKV7_GN(T, V, 4, 1) WKV7_GN(T, V, 8, 1) WKV7_GN(T, V, 16, 1) WKV7_GN(T, V, 32, 1)          \
    WKV7_GN(T, V, 64, 1) WKV7_GN(T, V, 64, 2) WKV7_GN(T, V, 128, 2) WKV7_GN(T, V, 256, 2)      \
    WKV7_GN(T, V, 512, 2) WKV7_GN(T, V, 256, 0)
    if (p.bf16) {
        WKV7_GN_ALL(bf16_t, 8)
        WKV7_GN_ALL(bf16_t, 2)
        WKV7_GN_ALL(bf16_t, 1)
    } else {
        WKV7_GN_ALL(float, 4)
        WKV7_GN_ALL(float, 1)
    }
    return hipErrorInvalidValue;
#undef WKV7_GN
#undef WKV7_GN_ALL
