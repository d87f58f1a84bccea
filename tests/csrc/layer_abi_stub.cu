// The argument checks of the head norm and cross attention (csrc/layer_abi.cu) without the
// kernels behind them: a launch is counted and succeeds, and every address is memory of the
// device but one that the test names.  So a call that passes all checks returns KATA_OK
// without a GPU, and one that is refused is refused by the check it is meant for.
#include "../../kernelized_linear_attention_fwd_b200/csrc/layer_abi.cu"

static const void *g_foreign = nullptr;
static int g_launches = 0;

namespace kata {
bool device_ptrs_ok(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (p && p == g_foreign) return false;
    return true;
}
dim3 norm_rotate_grid(const NormRotate &) { return dim3(7, 3); }
cudaError_t launch_norm_rotate(const NormRotate &, cudaStream_t) { return ++g_launches, cudaSuccess; }
cudaError_t launch_cross_forward(const CrossPlan &, const CrossIo &, cudaStream_t) { return ++g_launches, cudaSuccess; }
cudaError_t launch_cross_backward(const CrossPlan &, const CrossIo &, cudaStream_t) { return ++g_launches, cudaSuccess; }
}  // namespace kata

extern "C" {
void stub_foreign(const void *p) { g_foreign = p; }
int stub_launches() { return g_launches; }
}
