// The cut of a sum's steps into parts, one a workgroup.  Plain C++: the kernels use it and a host
// compiler takes it alone.
#pragma once

#include <stdint.h>

namespace glu {

// First step of part `part` when `steps` steps are cut into `parts` parts as even as whole steps
// allow: floor(steps part / parts), formed from the quotient and the remainder, since
// steps part itself passes 32 bits (2^25 steps of 64 rows, 256 parts).  Part `parts` is the end.
constexpr uint32_t part_begin(uint32_t steps, uint32_t part, uint32_t parts) {
  return steps / parts * part + steps % parts * part / parts;
}

}  // namespace glu
