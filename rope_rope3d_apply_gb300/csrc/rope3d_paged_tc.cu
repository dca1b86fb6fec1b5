// rope3d_paged_tc.cu -- the attention over pages for many rows on the tensor cores.
// (Not there yet: every call takes the kernel for few rows.)
#include "rope3d_paged.cuh"

namespace rope3d_paged {

int launch_tiles(const AttnParams &, const rope3d_paged_attention_args &, cudaStream_t) { return ROPE3D_ERR_CUDA; }
bool tiles_fit(const rope3d_paged_attention_args &) { return false; }
int tiles_wait_timeouts(unsigned int *count, bool) {
    *count = 0;
    return 0;
}

}  // namespace rope3d_paged
