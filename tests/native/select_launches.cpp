// Host program: the launches of the blocks' selection and of the split attention over
// selected tiles (block_select.cu, selected_split.cu, compiled as they are) over stand-ins
// for the CUDA runtime calls that make them.  It prints, for each call in turn, the limits
// that are set and the launches that are made, in their order:
//     limit kernel bytes
//     launch kernel ctas threads bytes cluster
// and behind those of a call what it was and gave:
//     select head_dim width group result
//     split head_dim heads items tokens partition taken result
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
    DecodeParams a = {};
    a.num_kv_heads = 1;
    a.block_size = 16;
    a.num_blocks = 1 << 20;
    for (int dim : {64, 128})
        for (int heads : {1, 4, 5, 8, 9})
            for (int items : {1, 8, 36, 37, 38, 72, 74, 75, 76, 200})
                for (int tokens : {32, 1024, 2048, 2064, 4096, 4112, 8192, 8208})
                    for (int partition : {16, 128, 512, 2048}) {
                        a.head_dim = dim;
                        a.num_heads = heads;
                        a.num_seqs = items;
                        a.max_blocks = tokens / 16;
                        a.partition_tokens = partition;
                        a.max_partitions = (tokens + partition - 1) / partition;
                        cudaError_t e = cudaSuccess;
                        const bool taken = selected_split(a, PKV_BF16, nullptr, &e);
                        std::printf("split %d %d %d %d %d %d %d\n", dim, heads, items, tokens,
                                    partition, (int)taken, (int)e);
                    }
    return 0;
}
