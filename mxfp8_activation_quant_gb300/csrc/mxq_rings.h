// How many panels of rows the attention's rings may have: the arithmetic, for host and device.
//
// Loads of panels land in any order, and the two sets of warps that take panels by turns wait only for their own. A wait by
// parity for a slot's use n passes while use n - 1 has not landed yet, so a set must know by other means that it has:
//  - in a ring of an even number of slots a slot is always the same set's, which has waited for its use n - 1 itself;
//  - else, by the chunks (one or two a panel) that a set has put into `chunks` slots of tensor memory. They are used up in order,
//    so the set that filled the last of panel q - 2 knows that everything `chunks` chunks before has landed: panel q - slots
//    has if the slots - 1 panels up to q - 2 have more chunks than that, which they have with slots >= chunks + 2.
#pragma once

namespace mxq {

constexpr bool ring_ok(int slots, int chunks) { return slots % 2 == 0 || slots >= chunks + 2; }
// The values' part of `slots`, where keys and values have rings of their own (the scores' thread waits for every panel of the keys):
// about half, an even number.
constexpr int value_ring(int slots) { return (slots / 2 + 1) & ~1; }
// The buffers of scales. With one panel a tile a set waits for its own tiles' alone, every second one; but one warp fills the buffers in
// order, so a set that has waited for tile n - 2 knows that tile n - bufs is there, odd or even.
constexpr bool scale_ring_ok(int bufs) { return bufs >= 2; }

}  // namespace mxq
