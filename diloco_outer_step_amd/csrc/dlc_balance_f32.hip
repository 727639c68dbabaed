// The balance loss over logits of type float.
#include "dlc_balance.h"

namespace dlc {

template <>
hipError_t launch_balance_of<kF32>(const BalanceArgs& a, bool one, hipStream_t s) {
  return launch_typed<float>(a, one, s);
}

}  // namespace dlc
