// pa_copy.cu -- copies of physical blocks in every layer's pool (copy-on-write
// after a fork, compaction; "11. 推理加速(一):vLLM 原理", §11.2: a shared block
// that would be written gets a copy first).
//
// A block is one contiguous run of num_kv_heads * block_size * head_dim
// elements in each of a layer's two arrays, so a pair is two plain copies per
// layer: nothing but HBM traffic, each byte read once and written once.  One
// 16-byte piece per thread and step keeps enough loads in flight: 58 blocks in each
// of 32 layers (243 MB read and written) take 37.5 us, 6.5 TB/s, 0.97 of the measured
// copy bandwidth; 2048 blocks in 8 layers (2.1 GB) 328 us, 0.98; 4 blocks in one layer
// 1.8 us, which is the launch.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {

// Grid-stride over the 16-byte pieces of all (pair, layer, K or V) copies.
__global__ void __launch_bounds__(256)
    copy_blocks_kernel(const CopyLayers arrays, int num_arrays, const int32_t *__restrict__ pairs,
                       int64_t total, int pieces_per_block, int num_blocks, unsigned *status) {
    pdl_wait();  // the pairs and the blocks may come from the previous kernel
    pdl_trigger();
    const int64_t per_pair = static_cast<int64_t>(num_arrays) * pieces_per_block;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t pair = i / per_pair;
        const int rem = static_cast<int>(i - pair * per_pair);
        const int a = rem / pieces_per_block, piece = rem - a * pieces_per_block;
        const int src = __ldg(pairs + 2 * pair), dst = __ldg(pairs + 2 * pair + 1);
        if (src < 0 || dst < 0 || src == dst) continue;
        if (src >= num_blocks || dst >= num_blocks) {
            flag_status(status, PA_DEV_BAD_BLOCK);
            continue;
        }
        uint4 *base = static_cast<uint4 *>(arrays.p[a]);
        base[static_cast<int64_t>(dst) * pieces_per_block + piece] =
            base[static_cast<int64_t>(src) * pieces_per_block + piece];
    }
}

int launch_copy_blocks(const pa_kv_desc *kv, int num_layers, const int32_t *pairs, int num_pairs,
                       int sms, unsigned *status, cudaStream_t s) {
    const int pieces = kv->num_kv_heads * kv->block_size * kv->head_dim *
                       (kv->kv_dtype == PA_KV_FP8_E4M3 ? 1 : 2) / 16;
    for (int l0 = 0; l0 < num_layers; l0 += kCopyLayers) {
        const int n = std::min(kCopyLayers, num_layers - l0);
        CopyLayers arrays{};
        for (int l = 0; l < n; ++l) {
            arrays.p[2 * l] = kv[l0 + l].k_cache;
            arrays.p[2 * l + 1] = kv[l0 + l].v_cache;
        }
        const int64_t total = static_cast<int64_t>(num_pairs) * 2 * n * pieces;
        const int64_t blocks = std::min<int64_t>((total + 255) / 256, 8 * static_cast<int64_t>(sms));
        PdlLaunch launch(static_cast<unsigned>(blocks), 256, 0, s);
        if (launch_kernel(launch, copy_blocks_kernel, arrays, 2 * n, pairs, total, pieces,
                          kv->num_blocks, status) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // namespace pa
