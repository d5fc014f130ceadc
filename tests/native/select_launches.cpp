// Host program: the launches of the blocks' selection and of the split attention over
// selected tiles (block_select.cu, selected_split.cu, compiled as they are) over stand-ins
// for the CUDA runtime calls that make them.  It prints, for each call in turn, the limits
// that are set and the launches that are made, in their order:
//     limit kernel bytes
//     launch kernel ctas threads bytes cluster
#include <cuda_runtime.h>

#include <cstdio>
#include <map>

#include "pkv.h"
#include "pkv_kernels.h"

namespace {

std::map<const void*, int> kernels;  // numbered as they come

int number(const void* kernel) { return kernels.emplace(kernel, (int)kernels.size()).first->second; }

}  // namespace

extern "C" {
cudaError_t cudaFuncSetAttribute(const void* kernel, cudaFuncAttribute attribute, int value)
{
    if (attribute == cudaFuncAttributeMaxDynamicSharedMemorySize)
        std::printf("limit %d %d\n", number(kernel), value);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* kernel, void**)
{
    int cluster = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension)
            cluster = (int)c->attrs[i].val.clusterDim.x;
    std::printf("launch %d %u %u %zu %d\n", number(kernel), c->gridDim.x, c->blockDim.x,
                c->dynamicSmemBytes, cluster);
    return cudaSuccess;
}
}

int main()
{
    SelectParams s = {};
    s.num_blocks = 1 << 20;
    s.block_size = 16;
    s.block_shift = 4;
    s.max_selected = 4;
    s.first_blocks = s.recent_blocks = 1;
    s.dtype = PKV_BF16;
    for (int dim : {64, 128})
        for (int width : {5, 64, 512, 513, 2048, 10000})
            for (int group : {1, 8, 9, 16, 28, 32, 64, 100, kSelectMaxGroup}) {
                s.num_seqs = 3;
                s.num_kv_heads = 2;
                s.num_heads = 2 * group;
                s.max_blocks = width;
                std::printf("select %d %d %d %d\n", dim, width, group,
                            (int)launch_select_blocks(s, dim, nullptr));
            }
    return 0;
}
