// What a matrix product reads and how it is cut into tiles, by sizes and types:
// plain arithmetic, without the device.
#pragma once

#include <cstdint>

namespace st {

// Bytes that may be read from the first of `rows` rows' scale bytes on, `stride`
// apart, of `blocks` blocks each: behind the last row's words there need not be
// anything (columns of a wider buffer end with it).  Words: scales lie on a grid of
// four bytes, so that the last one's rest is in the same page.
constexpr int scale_span(int rows, int stride, int blocks) { return (rows - 1) * stride + (blocks + 3) / 4 * 4; }

}  // namespace st
