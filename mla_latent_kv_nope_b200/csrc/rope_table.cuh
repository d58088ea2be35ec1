// Rotation of one position by a rope table (mla_rope_table): the angle of pair
// k at position p is p * turn[k] / 2^64 turns.  The product is formed modulo
// 2^64, so the fraction of a turn is exact at any position (a float or even a
// reduced double product would lose it at far ones); its top 32 bits, signed,
// are the angle over pi in [-1, 1) that sincospif takes.
#pragma once

#include "common.cuh"

namespace mla {

__device__ __forceinline__ void rope_turn_cos_sin(uint64_t turn, int64_t pos, float amplitude,
                                                  float* c, float* s) {
  const uint64_t f = turn * uint64_t(pos) + 0x80000000ull;   // rounded to 32 bits below
  const float x = float(int32_t(uint32_t(f >> 32))) * 4.656612873077393e-10f;   // * 2^-31
  float sn, cs;
  sincospif(x, &sn, &cs);
  *c = cs * amplitude;
  *s = sn * amplitude;
}

}  // namespace mla
