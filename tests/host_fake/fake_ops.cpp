// Test double of the operators' launchers, beside fake_device.cpp: the page
// calls act on host memory, attention and log probabilities do nothing.
#include <hip/hip_runtime_api.h>

#include <cstring>

#include "../../ragged_input_compilation_amd/csrc/ric_internal.h"

namespace ric {

hipError_t launch_page_copy(const PageParams& p, hipStream_t) {
    for (int l = 0; l < p.num_layers; ++l)
        for (const uint8_t* c : {p.kc[l], p.vc[l]})
            for (int k = 0; k < p.num_pairs; ++k)
                std::memmove(const_cast<uint8_t*>(c) + (int64_t)p.pairs[2 * k + 1] * p.block_bytes,
                             c + (int64_t)p.pairs[2 * k] * p.block_bytes, (size_t)p.block_bytes);
    for (int r = 0; r < p.rows; ++r)
        for (int j = 0; j < p.num_blocks[r]; ++j)
            for (int k = 0; k < p.num_pairs; ++k)
                if (p.blocks[r * p.blk_stride + j] == p.pairs[2 * k]) {
                    p.blocks[r * p.blk_stride + j] = p.pairs[2 * k + 1];
                    break;
                }
    return hipSuccess;
}

hipError_t launch_block_refs(const int32_t* blocks, int64_t blk_stride, const int32_t* num_blocks, int32_t rows,
                             int32_t pool, int32_t* refs, hipStream_t) {
    std::memset(refs, 0, (size_t)pool * 4);
    for (int r = 0; r < rows; ++r)
        for (int j = 0; j < num_blocks[r]; ++j) ++refs[blocks[r * blk_stride + j]];
    return hipSuccess;
}

hipError_t launch_fork(const ForkParams& p, bool rows, hipStream_t) {
    const int64_t page = (int64_t)p.block_size * p.row_bytes;
    for (int l = 0; l < p.num_layers; ++l)
        for (uint8_t* c : {p.kc[l], p.vc[l]})
            std::memmove(c + p.tail_block * page, c + p.blocks[p.parent * p.blk_stride + p.num_shared] * page,
                         (size_t)p.tail_rows * p.row_bytes);
    if (!rows) return hipSuccess;
    std::memcpy(p.tokens + p.child * p.tok_stride, p.tokens + p.parent * p.tok_stride, (size_t)p.num_tokens * 4);
    std::memcpy(p.blocks + p.child * p.blk_stride, p.blocks + p.parent * p.blk_stride, (size_t)p.num_shared * 4);
    return hipSuccess;
}

size_t attention_workspace(const AttnParams&) { return 0; }
hipError_t launch_attention(const AttnParams&, void*, hipStream_t) { return hipSuccess; }
size_t logprobs_workspace(int32_t, int32_t, int32_t) { return 0; }
size_t logprobs_workspace_up_to(int32_t, int32_t, int32_t) { return 0; }
hipError_t launch_logprobs(const LogprobParams&, void*, hipStream_t) { return hipSuccess; }

}  // namespace ric
