// attention_chunk_nvfp4.cu -- attention_chunk.cuh for one cache format (a
// translation unit per format, compiled in parallel).
#include "attention_chunk.cuh"

namespace nvfp4 {
namespace attn {

cudaError_t launch_chunk_nvfp4(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream)
{
    return chunk::launch_format<NVFP4_KV_NVFP4>(c, head_dim, workspace, num_sms, stream);
}

}  // namespace attn
}  // namespace nvfp4
