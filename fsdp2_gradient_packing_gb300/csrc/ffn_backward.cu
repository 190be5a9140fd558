#include "ffn_product.h"

namespace fsdp {
namespace ffn {

cudaError_t launch_backward(bool pair, Args &a, int sms, cudaStream_t stream) {
  return launch_columns(pair, a, sms, stream);
}

}  // namespace ffn
}  // namespace fsdp
