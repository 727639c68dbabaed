// The balance loss over logits of type __bf16.
#include "dlc_balance.h"

namespace dlc {

template <>
hipError_t launch_balance_of<kBF16>(const BalanceArgs& a, bool one, hipStream_t s) {
  return launch_typed<__bf16>(a, one, s);
}

}  // namespace dlc
