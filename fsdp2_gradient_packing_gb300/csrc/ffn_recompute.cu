#include "ffn_product.h"

namespace fsdp {
namespace ffn {

cudaError_t launch_recompute(bool pair, Args &a, int sms, cudaStream_t stream) {
  return launch_gated<RECOMPUTE>(pair, a, sms, stream);
}

}  // namespace ffn
}  // namespace fsdp
