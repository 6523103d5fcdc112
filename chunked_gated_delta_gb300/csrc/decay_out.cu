// decay_out.cu -- prompts of linear attention with a decay per head: the scan with its output.
#include "decay_scan.cuh"

namespace kda {

cudaError_t launch_decay_out(const DecayScanArgs& a, int K, int V, bool f16, cudaStream_t s) {
    return launch_scan_any<true>(a, K, V, f16, 1, s);
}

}  // namespace kda
