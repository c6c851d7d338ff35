// mx4_scales.hpp -- where a row's scales lie in LDS (mx4_a4w4.hip); plain C++, so that
// the places can be checked on the host.
//
// A row (or channel) of a tile has 16 bytes, the four words of scales of 512 K; a stage
// of 256 K uses two of them, read as eight bytes.  Where a row's words come by one load
// of 16 bytes, the load of its last 512 K ends with its last word, so the words lie
// `late` bytes further on than their number says.  With an odd number of words the last
// stage has one alone, at byte 12: its eight bytes take in the next row's first word,
// which is unused then (late is not 0), and is what the cut stage clears for it.  Behind
// the last row there is room for that word.  (A form whose reads stay in their row, from
// byte 8 with the lone word picked out of them, took 308 us for 8192^3, this one 293.)
#pragma once

namespace qp {

constexpr int kMxScaleRow = 16;
constexpr int kMxScaleRoom = 16;  // behind the last row; four bytes are used

// The word of scales that stage s's 512 K end before, and the bytes that a row of `words`
// lacks of the last ones: those words lie that many bytes late.
constexpr int mx_scales_end(int s) { return (s >> 1) * 4 + 4; }
constexpr int mx_scales_over(int words) { return (words + 3) / 4 * 16 - words * 4; }
// The byte from a row's first on where stage s's eight lie (where they are not late).
constexpr int mx_scales_at(int s) { return (s & 1) * 8; }

}  // namespace qp
