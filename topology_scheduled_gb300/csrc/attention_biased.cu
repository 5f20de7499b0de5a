// attention_biased.cu -- the forward kernel of attention_kernel.cuh, with a bias by buckets of the distance.
#include "attention_kernel.cuh"

namespace tsa {

tsa_status launch_biased_attention(const AttnLaunch &a, const BiasTerms &terms) {
    return launch_attention(a, terms);
}

}  // namespace tsa
