/* Stands in for the CUDA runtime calls of moe_expert_create on a machine without a GPU,
 * loaded before the library: they succeed, and note the kernels that are opted in to
 * their shared memory. One kernel's call can be made to fail. */
#include <cuda_runtime_api.h>

static const void *opted[1024];
static int count;
static const void *refused;

int fake_opted(const void **out) {
  for (int i = 0; i < count; ++i) out[i] = opted[i];
  const int n = count;
  count = 0;
  return n;
}
void fake_refuse(const void *kernel) { refused = kernel; }

cudaError_t cudaFuncSetAttribute(const void *f, enum cudaFuncAttribute attr, int value) {
  (void)attr, (void)value;
  if (f == refused) return cudaErrorInvalidDeviceFunction;
  if (count < 1024) opted[count++] = f;
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes *a, const void *f) {
  (void)f;
  a->numRegs = 255;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int *device) {
  *device = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *value, enum cudaDeviceAttr attr, int device) {
  (void)attr, (void)device;
  *value = 152;
  return cudaSuccess;
}
cudaError_t cudaMemset(void *p, int value, size_t bytes) {
  (void)p, (void)value, (void)bytes;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t stream) {
  (void)stream;
  return cudaSuccess;
}
