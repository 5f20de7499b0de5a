// attention.cu -- the forward kernel of attention_kernel.cuh, the scheduled attention itself.
#include "attention_kernel.cuh"

namespace tsa {

tsa_status launch_scheduled_attention(const AttnLaunch &a) {
    return launch_attention(a, NoTerms{});
}

}  // namespace tsa
