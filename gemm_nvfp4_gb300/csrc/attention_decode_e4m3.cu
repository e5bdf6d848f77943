// attention_decode_e4m3.cu -- attention_decode.cuh for one cache format (a
// translation unit per format, compiled in parallel).
#include "attention_decode.cuh"

namespace nvfp4 {
namespace attn {

cudaError_t launch_decode_e4m3(const Call &c, int head_dim, void *workspace, int num_sms, cudaStream_t stream)
{
    return decode::launch_format<NVFP4_KV_E4M3>(c, head_dim, workspace, num_sms, stream);
}

}  // namespace attn
}  // namespace nvfp4
