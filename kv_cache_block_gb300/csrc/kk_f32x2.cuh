// Two float32 operations in one instruction.
#pragma once

namespace kk {

#define KK_F32X2(name, op)                                                                       \
  __device__ __forceinline__ float2 name(float2 x, float2 y) {                                   \
    float2 r;                                                                                    \
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t" op          \
        " c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"                                                 \
        : "=f"(r.x), "=f"(r.y)                                                                   \
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));                                               \
    return r;                                                                                    \
  }
KK_F32X2(add2, "add.rn.f32x2")
KK_F32X2(sub2, "sub.rn.f32x2")
KK_F32X2(mul2, "mul.rn.f32x2")
#undef KK_F32X2
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ void set2(float* p, float2 x) { p[0] = x.x, p[1] = x.y; }

}  // namespace kk
