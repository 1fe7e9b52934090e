// A ring of stages as the row kernels drive it, on the host: one barrier a stage,
// copies that arrive in order until one does not, waits that then give up.  Exits
// with 1 where, at the end, a drain would not wait for a copy still in flight, or
// would wait for one that has arrived.
#include <cstdio>
#include <vector>

#include "ring_cursor.h"

using namespace moe;

struct Stage {
    int sent = 0, done = 0;                              // copies
    bool passed(uint32_t parity) const { return (uint32_t)(done & 1) != parity; }   // a try_wait's answer
};

// rows of one CTA; the copy of row `lost` does not arrive while the rows are worked
// on, nor does any after it; look = how many rows ahead a row's last barrier waits
static bool run(int rows, int stages, int lost, int look) {
    std::vector<Stage> st(stages);
    RingCursor c{stages};
    bool abort = false;
    int stop = rows;                                     // rows from it on are not sent for
    auto issue = [&](int row, int s) {
        ++st[s].sent;
        if (row < lost) ++st[s].done;
    };
    auto wait = [&](int t, int s, uint32_t parity) {     // while row t is worked on
        if (st[s].passed(parity)) return;
        abort = true;
        if (t + stages < stop) stop = t + stages;
    };
    for (int i = 0; i < stages && i < rows; ++i) issue(i, i);
    wait(0, 0, 0);
    if (look == 2 && rows > 1) wait(0, c.ahead(1), c.phase_ahead(1));
    for (int t = 0; t < rows; ++t, c.next()) {
        if (t + look < rows) wait(t, c.ahead(look), c.phase_ahead(look));
        if (t + stages < stop) issue(t + stages, c.slot);
    }
    if (lost < rows && !abort) return false;             // the model itself: the loss is noticed
    if (!abort) return true;
    for (int s = 0; s < stages && s < stop; ++s) {
        if (st[s].sent != (stop - 1 - s) / stages + 1) return false;
        const uint32_t parity = last_parity(stop, stages, s);
        if (st[s].passed(parity) != (st[s].done == st[s].sent)) return false;
        Stage late = st[s];
        late.done = late.sent;
        if (!late.passed(parity)) return false;          // the copies that come late end it
    }
    for (int s = stop; s < stages; ++s)
        if (st[s].sent) return false;
    return true;
}

int main() {
    int bad = 0;
    for (int stages = 3; stages <= 8; ++stages)
        for (int rows = 1; rows <= 40; ++rows)
            for (int lost = 0; lost <= rows; ++lost)
                for (int look = 1; look <= 2; ++look)
                    if (!run(rows, stages, lost, look) && ++bad <= 5)
                        std::printf("rows %d stages %d lost %d look %d\n", rows, stages, lost, look);
    std::printf("%d bad\n", bad);
    return bad != 0;
}
