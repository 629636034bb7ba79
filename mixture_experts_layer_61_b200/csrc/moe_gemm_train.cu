// moe_gemm_train.cu -- the training step's grouped products that keep the
// forward GEMM's shape (features x tokens): the gate/up projections that keep
// their pre-activations, and the two gradients with respect to the tokens,
// which contract over the weights' output axis and so take the weights as an
// MN-major operand, as they lie in memory.
#include "moe_gemm_host.cuh"

namespace moe {

int launch_gemm_train(TrainGemm kind, const GemmLaunch& L, const GemmCtl& ctl, cudaStream_t stream) {
    using bf = __nv_bfloat16;
    DeviceInfo d;
    int rc = current_device(&d);
    if (rc != 0) return rc;
    if (L.dtype != 0 || L.n_groups < 1 || L.n_groups > kMaxGroups || L.kdim <= 0 || L.n_out <= 0) return -1;
    if (L.x_rows <= 0) return 0;
    switch (kind) {
        case kTrainGateUp: return launch_variant<bf, bf, kEpiSwiGLUTrain, 256, 2>(L, ctl, d.num_sms, stream);
        case kTrainDownGrad: return launch_variant<bf, bf, kEpiSwiGLUGrad, 256, 2, true>(L, ctl, d.num_sms, stream);
        case kTrainGateUpGrad: return launch_variant<bf, bf, kEpiWide, 256, 2, true>(L, ctl, d.num_sms, stream);
    }
    return -1;
}

}  // namespace moe
