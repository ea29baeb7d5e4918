// Test-only: the decay tables' arithmetic of the decayed attention on its own, on the host and on the device.
#include "decay_unit.cuh"

namespace {
__global__ void decay_power_kernel(const float* g, const float* n, float* hi, float* lo, int count) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < count) gdn::decay_power(g[i], n[i], hi[i], lo[i]);
}
}  // namespace

extern "C" void decay_power_host(const float* g, const float* n, float* hi, float* lo, int count) {
    for (int i = 0; i < count; ++i) gdn::decay_power(g[i], n[i], hi[i], lo[i]);
}
extern "C" int decay_power_device(const float* g, const float* n, float* hi, float* lo, int count) {
    decay_power_kernel<<<(count + 255) / 256, 256>>>(g, n, hi, lo, count);
    return cudaDeviceSynchronize() == cudaSuccess ? 0 : 1;
}
