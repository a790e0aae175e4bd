#include "kernels.h"
namespace csa {
bool chunk_tc_supported(int, int, int, int, const csa_kv_cache&) { return false; }
size_t chunk_tc_workspace_bytes(int, int, int, int, int) { return 0; }
int chunk_tc_launch_count(int, int, int, int, int) { return 1; }
csa_status launch_chunk_attn_tc(const ChunkArgs&, const csa_kv_cache&, void*, size_t, cudaStream_t) { return CSA_ERR_UNSUPPORTED; }
}  // namespace csa
