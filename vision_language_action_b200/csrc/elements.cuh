// Loads of one element and stores of one or of 8 consecutive ones (16-byte
// accesses), fp32 or bf16 in memory and fp32 in registers (stores round to
// nearest even).
#pragma once

#include "common.cuh"

namespace svla {

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
