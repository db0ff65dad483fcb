// Loads and stores of 8 consecutive elements (16-byte accesses) or of one, fp32
// or bf16 in memory and fp32 in registers (stores round to nearest even).
#pragma once

#include "common.cuh"

namespace svla {

SVLA_DEV void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
SVLA_DEV void load8(const uint16_t* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
SVLA_DEV float load1(const float* p) { return *p; }
SVLA_DEV float load1(const uint16_t* p) { return bf2f(*p); }
SVLA_DEV void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
SVLA_DEV void store8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                            pack_bf16x2(x[6], x[7]));
}
SVLA_DEV void store1(float* p, float x) { *p = x; }
SVLA_DEV void store1(uint16_t* p, float x) {
  const __nv_bfloat16 b = __float2bfloat16_rn(x);
  *p = *reinterpret_cast<const uint16_t*>(&b);
}

}  // namespace svla
