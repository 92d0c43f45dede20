// Host state of libmoe_nvfp4.so shared by its entry points: the one-time
// preparation of each device and the tensor-map encoder.
#include <cudaTypedefs.h>

#include <mutex>

#include "host.h"
#include "kernels.h"
#include "train_kernels.h"
#include "w4a16_swap.h"

namespace moe {

namespace {

struct DeviceState {
    bool ready = false;
    moe_status status = MOE_ERR_UNSUPPORTED;
    int sms = 0;
};

std::mutex g_mu;
DeviceState g_dev[64];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

}  // namespace

moe_status device_state(int* sms, int* device) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState& d = g_dev[dev];
    if (!d.ready) {
        d.ready = true;
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            d.status = MOE_ERR_CUDA;
        } else if (major != 10 || minor != 3) {
            d.status = MOE_ERR_UNSUPPORTED;  // the binary carries sm_103a code only
        } else if (setup_routing_kernels() != cudaSuccess || setup_gemm_kernels() != cudaSuccess ||
                   setup_gemm_w4a16_kernels() != cudaSuccess || setup_gemm_pair_kernels(dev, d.sms) != cudaSuccess ||
                   setup_gemm_w4a16_pair_kernels(dev, d.sms) != cudaSuccess ||
                   setup_fused_layer_kernel() != cudaSuccess || setup_gemm_swap_kernels() != cudaSuccess ||
                   setup_gemm_w4a16_swap_kernels() != cudaSuccess ||
                   setup_router_gemm_kernel() != cudaSuccess ||
                   setup_expert_linear_kernels(dev, d.sms) != cudaSuccess ||
                   setup_layer_norm_kernels() != cudaSuccess || setup_sort_kernels() != cudaSuccess ||
                   setup_rms_norm_kernels() != cudaSuccess) {
            d.status = MOE_ERR_CUDA;
        } else {
            d.status = MOE_OK;
        }
        if (d.status == MOE_OK && g_encode == nullptr) {
            void* fn = nullptr;
            cudaDriverEntryPointQueryResult q;
            if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                    cudaSuccess ||
                q != cudaDriverEntryPointSuccess || fn == nullptr) {
                d.status = MOE_ERR_CUDA;
            } else {
                g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
            }
        }
    }
    *sms = d.sms;
    if (device) *device = dev;
    return d.status;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() { return g_encode; }

}  // namespace moe
