// Works out steps on the host (assign_plan.h).  In, for each step: n_tokens n_free listed
// page_shift max_pages n_seqs, then kv, keep and new lengths of each sequence; out:
// refused taken returned count left.
#include <cstdio>

#include "assign_plan.h"

int main()
{
    using namespace bevpool;
    AssignParams p{};
    int listed;
    while (scanf("%d %d %d %d %d %d", &p.n_tokens, &p.n_free, &listed, &p.page_shift, &p.max_pages, &p.n_seqs) == 6) {
        AssignSums all = {0, 0, 0};
        bool fits = true;
        for (int i = 0; i < p.n_seqs; ++i) {
            AssignGiven g;
            if (scanf("%d %d %d", &g.kv, &g.keep, &g.fresh) != 3) return 1;
            const AssignLengths l = lengths_of(p, g);
            fits &= l.fits;
            all = all + sums_of(l);
        }
        int64_t left;
        const AssignStep s = step_of(p, all, fits, listed, left);
        printf("%d %d %d %d %lld\n", s.refused, s.taken, s.returned, s.count, (long long)left);
    }
    return 0;
}
