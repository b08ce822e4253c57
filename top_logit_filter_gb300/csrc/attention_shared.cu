// The tensor-memory kernel for requests that share a prefix: the launches of
// topkp_shared_attention (attention.cu plans and joins them).
#include "attention_launch.cuh"

namespace topkp {

cudaError_t launch_grouped(const AttnDev& front, const AttnDev& own, cudaStream_t s) {
  Maps maps;
  const cudaError_t e = launch_parts<true>(front, maps, s);
  return e != cudaSuccess ? e : launch_parts<true>(own, maps, s);
}

cudaError_t grouped_take_device_error(unsigned int* out) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_error, sizeof(*out));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(zero));
  return e;
}

}  // namespace topkp
