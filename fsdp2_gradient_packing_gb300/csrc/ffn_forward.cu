#include "ffn_product.h"

namespace fsdp {
namespace ffn {

cudaError_t launch_forward(bool pair, Args &a, int sms, cudaStream_t stream) {
  return launch_gated<FORWARD>(pair, a, sms, stream);
}

}  // namespace ffn
}  // namespace fsdp
