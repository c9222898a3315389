// How the three products (Gram, square, update) of stacks are cut: "batch rows cols" triples on the
// command line, a line each.
#include "orth_plan.h"
#include <stdio.h>
#include <stdlib.h>
using namespace zk;
int main(int c, char** v) {
    static const char* nm[] = {"few", "mid", "two", "wide"};
    for (int i = 1; i + 2 < c; i += 3) {
        const int64_t B = atoll(v[i]), R = atoll(v[i + 1]), C = atoll(v[i + 2]);
        const OrthShape s = shape_of(B, R, C);
        const int64_t g = turns_of(R > C ? s.Rp : s.Cp), q = turns_of(s.m), n = s.group;
        const struct { OrthPlan p; int64_t tiles; } o[3] = {
            {plan_of(n, s.m, s.m, g, true, s.may_split), n * tiles_of(s.m, s.m, 256, true)},
            {plan_of(n, s.m, s.m, q, true, s.may_split), n * tiles_of(s.m, s.m, 256, true)},
            {plan_of(n, s.Rp, s.Cp, q, false, s.may_split), n * tiles_of(s.Rp, s.Cp, 256, false)}};
        printf("%lld %lld %lld", (long long)B, (long long)R, (long long)C);
        for (int k = 0; k < 3; ++k) {
            const int32_t left = (int32_t)o[k].p.split;
            printf(" %s%s%s%s", nm[o[k].p.kind], left ? "+split" : "", left && slices_of(left).r > 0 ? "+two" : "",
                   left && o[k].tiles > left ? "+whole" : "");
        }
        printf("\n");
    }
}
