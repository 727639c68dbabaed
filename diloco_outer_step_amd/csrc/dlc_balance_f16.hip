// The balance loss over logits of type _Float16.
#include "dlc_balance.h"

namespace dlc {

template <>
hipError_t launch_balance_of<kF16>(const BalanceArgs& a, bool one, hipStream_t s) {
  return launch_typed<_Float16>(a, one, s);
}

}  // namespace dlc
