// Words that workgroups of one launch hand each other through memory that is not
// cleared first: 16 bits of a value below 48 bits that belong to this launch
// alone, so that nothing left there can pass for it.
//
// The upper 32 bits, and seven of the next 16, count the launches of the process
// (2^39 of them, over all streams, devices and workspaces); the other nine of
// those 16 are the sign and exponent of a float32 or bf16 infinity or NaN, which
// no finite value of another call's scratch data has there. A launch that is
// captured into a graph keeps its number in every replay: its words are cleared
// by a kernel before it.
#pragma once

#include <cstdint>

namespace qlora {

constexpr uint64_t exchange_mark(uint64_t launch) {
  return (launch & 0xffffffffu) << 32 | (uint64_t)(0xff80u | (uint32_t)(launch >> 32 & 0x7fu)) << 16;
}
// (constexpr functions run on the device too)
constexpr uint64_t exchange_word(uint64_t mark, uint32_t bits) { return mark | (bits & 0xffffu); }
constexpr bool exchange_holds(uint64_t word, uint64_t mark) { return (word >> 16) == (mark >> 16); }

}  // namespace qlora
