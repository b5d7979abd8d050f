// The kind of tiles that each product with 4-bit weights takes, by the library's rules, on a card of 256
// compute units: lines "m T N K planes" and "e entries rows N K", one number a line out (-1: the few-row kernel).
#include <cstdio>

#include "../expert_cached_moe_amd/csrc/i4_plan.h"

int main() {
    using namespace moe::i4;
    char what;
    long long a, b, N, K;
    while (std::scanf(" %c", &what) == 1) {
        if (what == 'm') {
            if (std::scanf("%lld %lld %lld %lld", &a, &N, &K, &b) != 4) return 1;
            std::printf("%d\n", few_dense(a, N, K, 256) ? -1 : plan_dense(a, N, K, int(b), 256));
        } else {
            if (std::scanf("%lld %lld %lld %lld", &a, &b, &N, &K) != 4) return 1;
            std::printf("%d\n", plan_experts(int(a), b, N, K, 256));
        }
    }
    return 0;
}
