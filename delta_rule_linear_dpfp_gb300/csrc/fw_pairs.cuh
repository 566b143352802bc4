// fw_pairs.cuh -- packed fp32 pairs.
#pragma once

#include "fw_common.cuh"

namespace fw {

// Two floats that one instruction adds or multiplies (each rounded as the
// single instruction rounds it), for kernels near the instruction rate.
struct F2 {
    unsigned long long v;
};
FW_DEV F2 pack(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
FW_DEV float2 unpack(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
FW_DEV F2 both(float x) { return pack(x, x); }
FW_DEV F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
FW_DEV F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
FW_DEV F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
FW_DEV F2 operator-(F2 a, F2 b) { return fma2(b, both(-1.f), a); } // (one rounding)
// 2^x in one instruction (2^-22 of it; denormal results are 0).
FW_DEV float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
FW_DEV float sum(F2 a) {
    const float2 t = unpack(a);
    return t.x + t.y;
}

} // namespace fw
