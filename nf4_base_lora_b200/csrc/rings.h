// Which completed barrier phase frees a ring slot.  Plain constexpr functions, so
// that the kernels and a host check of the rule share them.
#pragma once

#include <cstdint>

namespace nf4lora {

// A wait for a phase's parity tells that phase from the ones next to it, but not
// from the one two before: it is sound only where the waiting thread itself knows
// that the phase before the awaited one is complete, and that the next one is not.
struct RingWait {
    int slot;         // of the ring whose barrier is waited on
    uint32_t parity;
};

// Step `it` (>= ds) of k_gemm's copies lands in decode slot it % ds, whose last
// user was step it - ds.  Its MMAs release that step's load slot too, and on the
// load ring's barriers the copying thread has waited for every earlier phase in
// turn (that of step it - ds - ls when it issued step it - ds); no later one can
// be complete, because step it - ds + ls >= it is not issued.  The decode ring's
// own barriers would not do: the thread has never waited on them, and with
// ls = 2 ds the phase before is that of step it - ls, of which it knows only that
// the other barrier's arrival has come.
constexpr RingWait decode_slot_release(int it, int ls, int ds) {
    return RingWait{(it - ds) % ls, static_cast<uint32_t>((it - ds) / ls) & 1u};
}

}  // namespace nf4lora
