// attention_differential.cu -- the forward kernel of attention_kernel.cuh, the difference of two softmax maps.
#include "attention_kernel.cuh"

namespace tsa {

tsa_status launch_differential_attention(const AttnLaunch &a, const DiffTerms &terms) {
    return launch_attention(a, terms);
}

}  // namespace tsa
