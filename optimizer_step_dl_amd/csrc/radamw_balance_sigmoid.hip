// radamw_balance_sigmoid.hip -- the rows of the balance loss for sigmoid scores
// (radamw_balance.h).
#include "radamw_balance.h"

namespace radamw {

hipError_t balance_rows_sigmoid(const BalanceArgs &a, const BalancePlan &p, bool sums, int dt, hipStream_t stream) {
    return balance_rows_of<true>(a, p, sums, dt, stream);
}

}  // namespace radamw
