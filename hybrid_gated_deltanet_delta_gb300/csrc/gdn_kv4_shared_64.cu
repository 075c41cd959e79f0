#include "gdn_kv4_attn.cuh"

namespace gdn {
namespace kv4 {

int shared_launch_64(const AttnArgs& a, int NT, int parts, cudaStream_t s) {
  return attn_launch_d<64, kShared>(a, NT, parts, s);
}

}  // namespace kv4
}  // namespace gdn
