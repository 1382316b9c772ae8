#include "sas_device.cuh"
#include "sas_kernels.h"
namespace sas {
void plan_chunk(ChunkParams& p) {}
size_t chunk_workspace_bytes(const ChunkParams& p) { return 0; }
void bind_chunk(ChunkParams& p, void* scratch) {}
cudaError_t launch_chunk(const ChunkParams& p, cudaStream_t stream) { return cudaErrorNotSupported; }
}
