// Soundness of decode_slot_release (csrc/rings.h) for the copying thread of
// k_gemm, whatever the barriers' arrivals are delayed by.
//
// A barrier with `done` completed phases lets a wait for parity P pass iff
// (done & 1) != P, phases being numbered from 0.  The copying thread issues steps
// in order; before step it >= LS it has waited for phase (it - LS) / LS of load
// barrier it % LS.  Steps complete in order and none completes before it is
// issued, but each barrier's arrival may come any time after that, so between two
// waits a barrier may have any count of completed phases from what the thread has
// itself seen there to what the issued steps allow.  For every extension step and
// every count that is possible then, the wait must pass iff step it - DS is
// complete, and must be able to pass.
//
// "dempty": the same for a wait on the decode ring's own barrier, which the check
// must find unsound at LS = 2 DS.
#include <cstdio>
#include <vector>

#include "rings.h"

using nf4lora::RingWait;

static int bad(int LS, int DS, int n_main, int n_ext, bool dempty) {
    int wrong = 0;
    std::vector<int> seen(LS, 0), dseen(DS, 0);  // completed phases the thread knows of
    const int n = n_main + n_ext;
    for (int it = 0; it < n; ++it) {
        if (it >= LS) seen[it % LS] = (it - LS) / LS + 1;
        if (it < n_main || it < DS) continue;
        const int s = it - DS;  // must be complete
        RingWait w;
        int need, low, high;
        if (dempty) {
            w = RingWait{it % DS, (static_cast<uint32_t>(it / DS) & 1u) ^ 1u};
            need = s / DS + 1;
            low = dseen[w.slot];
            high = need;  // step it is not issued
        } else {
            w = nf4lora::decode_slot_release(it, LS, DS);
            if (w.slot != s % LS) ++wrong;
            need = s / LS + 1;
            low = seen[w.slot];
            high = 0;  // of the issued steps on this barrier
            for (int q = w.slot; q < it; q += LS) ++high;
        }
        for (int done = low; done <= high; ++done)
            if (((done & 1) != static_cast<int>(w.parity)) != (done >= need)) ++wrong;
        if (dempty) dseen[w.slot] = need;
        else seen[w.slot] = need > seen[w.slot] ? need : seen[w.slot];
    }
    return wrong;
}

int main() {
    int wrong = 0, old_wrong = 0;
    for (int DS = 1; DS <= 6; ++DS)
        for (int LS = DS < 2 ? 2 : DS; LS <= 8; ++LS)
            for (int n_main = 1; n_main <= 40; ++n_main)
                for (int n_ext = 2; n_ext <= 8; n_ext += 2) {
                    wrong += bad(LS, DS, n_main, n_ext, false);
                    if (LS == 2 * DS) old_wrong += bad(LS, DS, n_main, n_ext, true);
                }
    std::printf("%d %d\n", wrong, old_wrong > 0);
    return 0;
}
