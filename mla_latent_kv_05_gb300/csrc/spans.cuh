// What a TMA tensor map may claim to span.
#pragma once
#include <cstdint>

namespace mla {

// TMA boxes from a tensor map that spans less than 128 KiB load about three
// times slower (a 100-row expansion took 30 us, a 128-row one 13 us, and the
// 100 rows with a wider stride 13 us).  So a map over such a tensor gets one more
// dimension of two entries, of which only entry 0 is ever addressed, where the
// memory that entry 1 would take is part of the same allocation: TMA may touch
// whatever a map claims.  (A map that claimed 16 MiB behind a tensor faulted where
// the tensor ended less than a box's rows before the end of the mapped memory.)
//
// Byte stride of entry 1 for a tensor of `bytes` at `base`: 0 where the map takes
// no second entry, because it is wide enough or because there is no room (its boxes
// then load at the slow rate).
uint64_t tma_far(const void* base, uint64_t bytes);

}  // namespace mla
