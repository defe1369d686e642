// Tree attention over fp16 caches on the tensor cores (tree_mma.cuh).
#include "tree_mma.cuh"

namespace pkv {

cudaError_t launch_tree_f16(int D, const TreeParams &p, cudaStream_t s) { return launch_rows<__half>(D, p, s); }

}  // namespace pkv
