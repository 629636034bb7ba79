// moe_gemm_train.cu -- the training step's grouped products that keep the
// forward GEMM's shape (features x tokens): the gate/up projections that keep
// their pre-activations, and the two gradients with respect to the tokens,
// which contract over the weights' output axis and so take the weights as an
// MN-major operand, as they lie in memory.  Single calls / back to back, at the
// clock the power cap leaves: Mixtral-shaped, T = 2048: gate/up with
// pre-activations 762 / 934 us, down gradient 428 / 536 us; Qwen2-MoE-shaped,
// T = 2048: 600 / 759 us and the token gradient 565 / 718 us.
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
        case kTrainGateUpGrad:
            // 512-feature tiles read 25 % fewer operand bytes; 256-feature ones where
            // those, cut into k-slices of at least 16 steps of 64, would not give
            // every SM pair work (8 experts of 1024 x 1024, 512 tokens: 37 us wide,
            // 33 us; Mixtral-shaped, 64 tokens: 268 us wide, 370 us).  The token rows
            // are not in the rule: few experts of many rows, whose row chunks would give
            // the wide tiles work enough, take the narrow ones too (not measured wide)
            if ((long long)L.n_groups * ((L.n_out + 511) / 512) * (L.kdim < 4096 ? (L.kdim + 1023) / 1024 : 4) <
                d.num_sms / 2)
                return launch_variant<bf, bf, kEpiPlain, 256, 2, true>(L, ctl, d.num_sms, stream);
            return launch_variant<bf, bf, kEpiWide, 256, 2, true>(L, ctl, d.num_sms, stream);
    }
    return -1;
}

}  // namespace moe
