// The classes of entries by which the log probabilities' alternatives are bounded
// (csrc/xent_units.h), on the host: the run ahead and the run over all entries
// together put every entry that has a class into one class only, and every entry
// has one.
#include "xent_units.h"

#include <cstdio>
#include <vector>

using namespace carbon;

int main() {
    int with = 0, without = 0;
    for (int64_t M : {257, 300, 1100, 8192})
        for (int64_t V : {300, 5003, 16383, 16384, 20001, 50257, 131072})
            for (int top : {1, 5, 8, 9, 14, 20, 28}) {
                Plan p;
                make_plan(&p, nullptr, M, 64, V, false, false, top);
                const int classes = top_classes(p.listed);
                if (p.piloted % kGroup != 0 || p.piloted > V || kGroup % kPilotBlock != 0) return 1;
                (p.piloted > 0 ? with : without) += 1;
                std::vector<int> of((size_t)V, -1);
                auto put = [&](int64_t from, int64_t n, int cls) {
                    if (cls < 0) return true;
                    if (cls >= classes) return false;
                    for (int64_t e = from; e < from + n && e < V; ++e) {
                        if (of[(size_t)e] >= 0) return false;         // in a class already
                        of[(size_t)e] = cls;
                    }
                    return true;
                };
                for (int64_t e = 0; e < p.piloted; e += kPilotBlock)
                    if (!put(e, kPilotBlock, pilot_class(p, (int)e))) return 2;
                for (int64_t e = 0; e < V; e += kGroup)
                    if (!put(e, kGroup, group_class(p, (int)e))) return 3;
                for (int cls : of)
                    if (cls < 0) return 4;
            }
    if (with < 50 || without < 50) return 5;
    std::puts("ok");
    return 0;
}
