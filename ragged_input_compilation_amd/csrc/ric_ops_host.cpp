// C entry points of the operators around the step: attention over the paged
// cache, log probabilities, and page copies, moves, counts and forks.  Argument
// checks and launches; the kernels are in ric_attention.hip, ric_logprobs.hip and
// ric_pages.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <utility>
#include <vector>

#include "../../include/ric.h"
#include "ric_batch.h"
#include "ric_internal.h"

using namespace ric;

namespace {

constexpr int32_t kMaxOperatorRows = 1 << 22;   // tokens or logits rows per call
constexpr int32_t kMaxVocab = 1 << 30;          // token ids and the strides over them stay below 2^31

int check_attention(const ric_attention* a, int32_t num_reqs, int32_t num_tokens, int32_t max_query_len,
                    int32_t max_seq_len, AttnParams* p) {
    if (!a) return fail(RIC_EINVAL, "attention description is NULL");
    if (a->dtype != RIC_F16 && a->dtype != RIC_BF16) return fail(RIC_EINVAL, "dtype %d is not RIC_F16 or RIC_BF16", a->dtype);
    if (a->num_heads < 1 || a->num_kv_heads < 1 || a->num_heads % a->num_kv_heads != 0)
        return fail(RIC_EINVAL, "num_heads %d is not a positive multiple of num_kv_heads %d", a->num_heads, a->num_kv_heads);
    if (a->num_heads > 512) return fail(RIC_EINVAL, "num_heads %d above 512", a->num_heads);
    if (a->head_dim < 8 || a->head_dim > 256 || a->head_dim % 8 != 0)
        return fail(RIC_EINVAL, "head_dim %d is not a multiple of 8 in [8, 256]", a->head_dim);
    if (a->block_size < 1) return fail(RIC_EINVAL, "block_size %d < 1", a->block_size);
    if (!std::isfinite(a->scale)) return fail(RIC_EINVAL, "scale is not finite");
    if (!(a->softcap >= 0.f) || !std::isfinite(a->softcap)) return fail(RIC_EINVAL, "softcap must be finite and >= 0");
    if (a->window < 0 || a->window > (1 << 30)) return fail(RIC_EINVAL, "window %d outside [0, 2^30]", a->window);
    if (num_reqs < 0 || num_tokens < 0) return fail(RIC_EINVAL, "negative count");
    if (num_tokens > kMaxOperatorRows) return fail(RIC_EINVAL, "num_tokens %d above %d per call", num_tokens, kMaxOperatorRows);
    // Grids stay below 2^24 workgroups of 256 lanes: a request's rows are cut into
    // tiles of 128, its keys into 16 pieces per K/V head (256 where requests are few).
    const int64_t tiles = ((int64_t)num_tokens * (a->num_heads / a->num_kv_heads) / 128 + num_reqs) * a->num_kv_heads;
    if (num_reqs > 65535 || (int64_t)num_reqs * a->num_kv_heads >= (1 << 20) || tiles >= kMaxRowsPerLaunch)
        return fail(RIC_EINVAL, "%d requests with %d tokens of %d heads are too many for one call", num_reqs, num_tokens, a->num_heads);
    if (max_query_len < 0 || max_seq_len < 0) return fail(RIC_EINVAL, "negative length");
    *p = AttnParams{};
    p->slopes = a->alibi_slopes;
    p->prefix = a->prefix_lens;
    p->num_reqs = num_reqs;
    p->num_tokens = num_tokens;
    p->max_q = std::min(max_query_len, num_tokens);
    p->max_seq = max_seq_len;
    p->heads = a->num_heads;
    p->kv_heads = a->num_kv_heads;
    p->dim = a->head_dim;
    p->block_size = a->block_size;
    p->block_shift = ilog2_exact(a->block_size);
    p->window = a->window;
    p->scale = a->scale;
    p->cap = a->softcap;
    p->bf16 = a->dtype == RIC_BF16;
    return RIC_OK;
}

// The pages of a call and what they are in it: open addressing over a table at
// most half full (1500 pairs: 141 us for the whole call, whose kernel takes 131;
// with sets that allocate a node per page the host took longer than that, 160).
enum PageRole { kSource = 0, kDestination = 1, kNew = 2 };
class PageSet {
  public:
    explicit PageSet(int32_t pairs) {
        while (bits_ < 32 && (int64_t(1) << bits_) < 4 * (int64_t)pairs) ++bits_;     // fewer than 2^31 ids exist
        table_.assign((size_t)1 << bits_, 0);
    }
    // Enters a page that is not there yet; what it was before.
    PageRole insert(int32_t page, PageRole role) {
        const size_t mask = table_.size() - 1;
        size_t at = ((uint32_t)page * 0x9E3779B1u) >> (32 - bits_);       // 2^32 / golden ratio: spreads runs of ids
        for (; table_[at] != 0; at = (at + 1) & mask)
            if ((table_[at] - 1) >> 1 == (uint32_t)page) return (PageRole)((table_[at] - 1) & 1);
        table_[at] = ((uint32_t)page << 1 | (uint32_t)role) + 1;
        return kNew;
    }

  private:
    int bits_ = 4;
    std::vector<uint32_t> table_;
};

// Checks shared by the page calls; resolves the group.
int check_pages(ric_batch* b, int32_t group, int32_t n, const int32_t* src, const int32_t* dst,
                void* const* k_cache, void* const* v_cache, int32_t num_layers, int64_t block_bytes, bool distinct_src) {
    if (group < 0 || group >= b->L.groups) return fail(RIC_EINVAL, "group %d outside [0, %d)", group, b->L.groups);
    if (n < 0 || num_layers < 0) return fail(RIC_EINVAL, "negative count");
    if (n > 0 && (!src || !dst)) return fail(RIC_EINVAL, "NULL pointer argument");
    if (num_layers > 0) {
        if (!k_cache || !v_cache) return fail(RIC_EINVAL, "NULL pointer argument");
        if (block_bytes <= 0 || block_bytes % 16 != 0 || block_bytes > (int64_t(1) << 31))
            return fail(RIC_EINVAL, "block_bytes %lld is not a positive multiple of 16 up to 2^31", (long long)block_bytes);
        for (int32_t l = 0; l < num_layers; ++l)
            if (!k_cache[l] || !v_cache[l] || !aligned16(k_cache[l]) || !aligned16(v_cache[l]))
                return fail(RIC_EINVAL, "layer %d: NULL or misaligned pointer", l);
    }
    int rc = check_blocks(b, group, src, n);
    if (rc) return rc;
    rc = check_blocks(b, group, dst, n);
    if (rc) return rc;
    try {
        PageSet pages(n);
        for (int32_t k = 0; k < n; ++k)
            if (pages.insert(src[k], kSource) != kNew && distinct_src)
                return fail(RIC_EINVAL, "page %d is listed twice as a source", src[k]);
        for (int32_t k = 0; k < n; ++k) {
            const PageRole was = pages.insert(dst[k], kDestination);
            if (was == kDestination) return fail(RIC_EINVAL, "page %d is listed twice as a destination", dst[k]);
            if (was == kSource) return fail(RIC_EINVAL, "page %d is both a source and a destination", dst[k]);
        }
    } catch (const std::bad_alloc&) {
        return fail(RIC_ENOMEM, "host allocation failed");
    }
    return RIC_OK;
}

int copy_pages(ric_batch* b, int32_t group, int32_t n, const int32_t* src, const int32_t* dst, void* const* k_cache,
               void* const* v_cache, int32_t num_layers, int64_t block_bytes, bool tables) {
    if (n == 0) return RIC_OK;
    int rc = refuse_if_capturing(b);
    if (rc) return rc;
    std::vector<std::pair<int32_t, int32_t>> pairs;
    try {
        pairs.resize((size_t)n);
    } catch (const std::bad_alloc&) {
        return fail(RIC_ENOMEM, "host allocation failed");
    }
    for (int32_t k = 0; k < n; ++k) pairs[k] = {src[k], dst[k]};
    if (tables) std::sort(pairs.begin(), pairs.end());
    // A 16-KiB piece of a page is one workgroup: fewer pairs per launch for
    // huge pages, so that the grid stays below 2^24 workgroups of 256 lanes.
    const int64_t pieces = num_layers > 0 ? (block_bytes + 16383) / 16384 : 1;
    const int32_t per_launch = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kMaxPagePairs, (kMaxRowsPerLaunch - 1) / pieces));
    for (int32_t k0 = 0; k0 < n; k0 += per_launch) {
        const int32_t m = std::min(per_launch, n - k0);
        rc = stage(b, b->d_pages, pairs.data() + k0, 2 * (size_t)m);
        if (rc) return rc;
        rc = flush(b);
        if (rc) return rc;
        int32_t l0 = 0;
        do {
            PageParams p{};
            p.num_layers = std::min<int32_t>(kMaxLayersPerLaunch, num_layers - l0);
            for (int i = 0; i < p.num_layers; ++i) {
                p.kc[i] = static_cast<const uint8_t*>(k_cache[l0 + i]);
                p.vc[i] = static_cast<const uint8_t*>(v_cache[l0 + i]);
            }
            p.pairs = b->d_pages;
            p.block_bytes = num_layers > 0 ? block_bytes : 16;
            p.num_pairs = m;
            if (tables && l0 == 0) {
                p.blocks = b->blk(group);
                p.num_blocks = b->dcol(blocks_col(group));
                p.blk_stride = b->bstride(group);
                p.rows = b->num_live;
            }
            HIP_TRY(launch_page_copy(p, b->stream));
            l0 += kMaxLayersPerLaunch;
        } while (l0 < num_layers);
    }
    return RIC_OK;
}

}  // namespace

extern "C" {

size_t ric_paged_attention_workspace_bytes(const ric_attention* a, int32_t num_reqs, int32_t num_tokens,
                                           int32_t max_query_len, int32_t max_seq_len) {
    AttnParams p;
    if (check_attention(a, num_reqs, num_tokens, max_query_len, max_seq_len, &p)) return 0;
    if (num_reqs == 0 || num_tokens == 0) return 0;
    return align_up(attention_workspace(p), kAlign);
}

int ric_paged_attention(const ric_attention* a, const void* q, int64_t q_stride, const void* k_cache,
                        const void* v_cache, int64_t num_blocks, const int32_t* block_table,
                        int64_t block_table_stride, int32_t block_table_width, const int32_t* query_start_loc,
                        const int32_t* seq_lens, int32_t num_reqs, int32_t num_tokens, int32_t max_query_len,
                        int32_t max_seq_len, void* out, int64_t out_stride, void* workspace,
                        size_t workspace_bytes, int32_t* dev_status, void* stream) {
    AttnParams p;
    int rc = check_attention(a, num_reqs, num_tokens, max_query_len, max_seq_len, &p);
    if (rc) return rc;
    const int64_t row = (int64_t)a->num_heads * a->head_dim * 2;
    if (q_stride == 0) q_stride = row;
    if (out_stride == 0) out_stride = row;
    if (q_stride < row || out_stride < row || q_stride % 16 != 0 || out_stride % 16 != 0)
        return fail(RIC_EINVAL, "q/out strides must be multiples of 16 and >= %lld", (long long)row);
    if (num_blocks < 1 || num_blocks * (int64_t)a->block_size >= (int64_t(1) << 31) || num_blocks >= (int64_t(1) << 31))
        return fail(RIC_EINVAL, "num_blocks %lld * block_size %d outside [1, 2^31)", (long long)num_blocks, a->block_size);
    if (block_table_width < 0 || block_table_stride < block_table_width)
        return fail(RIC_EINVAL, "block_table_width %d outside [0, stride %lld]", block_table_width, (long long)block_table_stride);
    if (num_reqs == 0 || num_tokens == 0) return RIC_OK;
    if (!q || !k_cache || !v_cache || !block_table || !query_start_loc || !seq_lens || !out)
        return fail(RIC_EINVAL, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return fail(RIC_EINVAL, "q, caches and out must be 16-byte aligned");
    const size_t need = attention_workspace(p);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return fail(RIC_EINVAL, "workspace of %zu bytes is NULL, misaligned or below the %zu needed", workspace_bytes, need);
    p.q = static_cast<const uint8_t*>(q);
    p.out = static_cast<uint8_t*>(out);
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.kc = static_cast<const uint8_t*>(k_cache);
    p.vc = static_cast<const uint8_t*>(v_cache);
    p.table = block_table;
    p.table_stride = block_table_stride;
    p.qsl = query_start_loc;
    p.seq = seq_lens;
    p.status = dev_status;
    p.num_blocks = num_blocks;
    p.table_width = block_table_width;
    HIP_TRY(launch_attention(p, workspace, static_cast<hipStream_t>(stream)));
    return RIC_OK;
}

size_t ric_token_logprobs_workspace_bytes(int32_t max_rows, int32_t vocab, int32_t top_k) {
    if (max_rows <= 0 || max_rows > kMaxOperatorRows || vocab < 1 || vocab > kMaxVocab || top_k < 0 || top_k > kMaxTopLogprobs)
        return 0;
    return align_up(logprobs_workspace_up_to(max_rows, vocab, top_k), kAlign);
}

int ric_token_logprobs(const void* logits, int32_t dtype, int64_t row_stride, const int32_t* targets,
                       const int32_t* dev_count, int32_t max_rows, int32_t vocab, int32_t top_k, float* logprob,
                       int32_t* rank, float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                       size_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (dtype != RIC_F16 && dtype != RIC_BF16 && dtype != RIC_F32) return fail(RIC_EINVAL, "unknown dtype %d", dtype);
    if (max_rows < 0 || max_rows > kMaxOperatorRows)
        return fail(RIC_EINVAL, "max_rows %d outside [0, %d]", max_rows, kMaxOperatorRows);
    if (vocab < 1 || vocab > kMaxVocab) return fail(RIC_EINVAL, "vocab %d outside [1, 2^30]", vocab);
    if (top_k < 0 || top_k > kMaxTopLogprobs || top_k > vocab)
        return fail(RIC_EINVAL, "top_k %d outside [0, min(%d, vocab)]", top_k, kMaxTopLogprobs);
    const int64_t size = dtype == RIC_F32 ? 4 : 2;
    if (row_stride == 0) row_stride = size * vocab;
    if (row_stride < size * vocab || row_stride % size != 0)
        return fail(RIC_EINVAL, "row_stride %lld must be a multiple of %lld and hold the row", (long long)row_stride, (long long)size);
    if (max_rows == 0) return RIC_OK;
    if (!logits || reinterpret_cast<uintptr_t>(logits) % size != 0) return fail(RIC_EINVAL, "logits are NULL or misaligned");
    if ((targets != nullptr) != (logprob != nullptr) || (targets != nullptr) != (rank != nullptr))
        return fail(RIC_EINVAL, "targets, logprob and rank come together");
    if ((top_k > 0) != (top_ids != nullptr) || (top_k > 0) != (top_logprobs != nullptr))
        return fail(RIC_EINVAL, "top_ids and top_logprobs come with top_k > 0");
    const size_t need = logprobs_workspace(max_rows, vocab, top_k);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return fail(RIC_EINVAL, "workspace of %zu bytes is NULL, misaligned or below the %zu needed", workspace_bytes, need);
    LogprobParams p{};
    p.logits = static_cast<const uint8_t*>(logits);
    p.row_stride = row_stride;
    p.targets = targets;
    p.dev_count = dev_count;
    p.logprob = logprob;
    p.rank = rank;
    p.entropy = entropy;
    p.top_ids = top_ids;
    p.top_logprobs = top_logprobs;
    p.status = dev_status;
    p.max_rows = max_rows;
    p.vocab = vocab;
    p.top_k = top_k;
    p.dtype = dtype;
    HIP_TRY(launch_logprobs(p, workspace, static_cast<hipStream_t>(stream)));
    return RIC_OK;
}

int ric_copy_blocks(ric_batch* b, int32_t group, int32_t n, const int32_t* src, const int32_t* dst,
                    void* const* k_cache, void* const* v_cache, int32_t num_layers, int64_t block_bytes) {
    if (!b) return fail(RIC_EINVAL, "handle is NULL");
    DeviceScope ds(b);
    int rc = check_pages(b, group, n, src, dst, k_cache, v_cache, num_layers, block_bytes, false);
    if (rc || num_layers == 0) return rc;
    return copy_pages(b, group, n, src, dst, k_cache, v_cache, num_layers, block_bytes, false);
}

int ric_move_blocks(ric_batch* b, int32_t group, int32_t n, const int32_t* src, const int32_t* dst,
                    void* const* k_cache, void* const* v_cache, int32_t num_layers, int64_t block_bytes) {
    if (!b) return fail(RIC_EINVAL, "handle is NULL");
    DeviceScope ds(b);
    int rc = check_pages(b, group, n, src, dst, k_cache, v_cache, num_layers, block_bytes, true);
    if (rc) return rc;
    if (b->used_rows() != b->num_live) return fail(RIC_ESTATE, "rows are not condensed");
    rc = copy_pages(b, group, n, src, dst, k_cache, v_cache, num_layers, block_bytes, true);
    if (rc) return rc;
    b->scheduled = false;      // compiled slots name the old pages
    return RIC_OK;
}

int ric_block_refs(ric_batch* b, int32_t group, int32_t* dev_refs) {
    if (!b) return fail(RIC_EINVAL, "handle is NULL");
    DeviceScope ds(b);
    if (group < 0 || group >= b->L.groups) return fail(RIC_EINVAL, "group %d outside [0, %d)", group, b->L.groups);
    if (!dev_refs) return fail(RIC_EINVAL, "dev_refs is NULL");
    if (b->used_rows() != b->num_live) return fail(RIC_ESTATE, "rows are not condensed");
    int rc = flush(b);
    if (rc) return rc;
    HIP_TRY(launch_block_refs(b->blk(group), b->bstride(group), b->dcol(blocks_col(group)), b->num_live,
                              group_pool(b->cfg, group), dev_refs, b->stream));
    return RIC_OK;
}

int ric_fork_request(ric_batch* b, uint64_t parent_id, uint64_t child_id, int32_t num_tokens, int32_t num_computed,
                     const int32_t* new_blocks, int32_t num_new, void* const* k_cache, void* const* v_cache,
                     int32_t num_layers, int32_t row_bytes, const ric_sampling* sampling, int32_t* out_row) {
    if (!b) return fail(RIC_EINVAL, "handle is NULL");
    DeviceScope ds(b);
    int32_t parent;
    int rc = find(b, parent_id, &parent);
    if (rc) return rc;
    if (b->row_of.count(child_id)) return fail(RIC_EEXIST, "request id %llu is live", (unsigned long long)child_id);
    const int32_t T = b->S(kNumTokens, parent), P = b->S(kNumPrompt, parent), B = b->cfg.block_size;
    if (num_tokens < P || num_tokens > T)
        return fail(RIC_ERANGE, "%d tokens outside [prompt %d, history %d] of the parent", num_tokens, P, T);
    if (num_computed < 0 || num_computed > num_tokens)
        return fail(RIC_ERANGE, "num_computed %d outside [0, %d]", num_computed, num_tokens);
    const int32_t shared = num_computed / B, tail = num_computed % B;
    if (shared + (tail > 0 ? 1 : 0) > b->S(kNumBlocks, parent))
        return fail(RIC_ERANGE, "the parent's %d blocks cannot hold %d computed tokens", b->S(kNumBlocks, parent), num_computed);
    if (num_new < 0 || (int64_t)shared + num_new > b->cfg.max_blocks_per_req)
        return fail(RIC_ERANGE, "%d shared + %d new blocks outside the table capacity %d", shared, num_new, b->cfg.max_blocks_per_req);
    if (tail > 0 && num_new < 1) return fail(RIC_EINVAL, "a partly filled page needs a new block");
    if ((num_new > 0 && !new_blocks) || num_layers < 0) return fail(RIC_EINVAL, "NULL or negative argument");
    rc = check_blocks(b, 0, new_blocks, num_new);
    if (rc) return rc;
    if (num_layers > 0) {
        if (!k_cache || !v_cache) return fail(RIC_EINVAL, "NULL pointer argument");
        if (row_bytes <= 0 || row_bytes % 16 != 0) return fail(RIC_EINVAL, "row_bytes %d not a positive multiple of 16", row_bytes);
        for (int32_t l = 0; l < num_layers; ++l)
            if (!k_cache[l] || !v_cache[l] || !aligned16(k_cache[l]) || !aligned16(v_cache[l]))
                return fail(RIC_EINVAL, "layer %d: NULL or misaligned pointer", l);
    }
    int32_t row = -1;
    for (int32_t r = 0; r < b->cfg.max_num_reqs && row < 0; ++r)
        if (!b->live[r]) row = r;
    if (row < 0) return fail(RIC_EFULL, "no free row (max_num_reqs %d)", b->cfg.max_num_reqs);
    rc = refuse_if_capturing(b);
    if (rc) return rc;
    rc = before_row_overwrite(b, row);
    if (rc) return rc;
    rc = stage(b, b->d_blk + (int64_t)row * b->L.blk_stride + shared, new_blocks, (size_t)num_new);
    if (rc) return rc;
    int32_t vals[kNumScalarCols] = {num_tokens, P, num_computed, 0, shared + num_new, b->S(kTopK, parent),
                                    b->S(kTemperature, parent), b->S(kTopP, parent), b->S(kRepPenalty, parent)};
    if (sampling) {
        vals[kTopK] = sampling->top_k;
        vals[kTemperature] = as_bits(sampling->temperature);
        vals[kTopP] = as_bits(sampling->top_p);
        vals[kRepPenalty] = as_bits(sampling->repetition_penalty);
    }
    for (int c = 0; c < kNumScalarCols; ++c) {
        b->S(c, row) = vals[c];
        b->mark(c, row);
    }
    b->live[row] = 1;
    b->req_at[row] = child_id;
    b->row_of[child_id] = row;
    b->pending_epoch[row] = b->epoch;
    ++b->num_live;
    b->scheduled = false;
    // The parent's staged tokens and pages land before the kernel reads them.
    rc = flush(b);
    if (rc) return rc;
    const int32_t copied = tail > 0 ? num_layers : 0;
    int32_t l0 = 0;
    do {
        ForkParams p{};
        p.num_layers = std::min<int32_t>(kMaxLayersPerLaunch, copied - l0);
        for (int i = 0; i < p.num_layers; ++i) {
            p.kc[i] = static_cast<uint8_t*>(k_cache[l0 + i]);
            p.vc[i] = static_cast<uint8_t*>(v_cache[l0 + i]);
        }
        p.row_bytes = copied > 0 ? row_bytes : 0;
        p.block_size = B;
        p.pool = b->cfg.num_kv_blocks;
        p.tokens = b->d_tok;
        p.tok_stride = b->L.tok_stride;
        p.blocks = b->d_blk;
        p.blk_stride = b->L.blk_stride;
        p.parent = parent;
        p.child = row;
        p.num_tokens = num_tokens;
        p.num_shared = shared;
        p.tail_rows = tail;
        p.tail_block = num_new > 0 ? new_blocks[0] : 0;
        HIP_TRY(launch_fork(p, l0 == 0, b->stream));
        l0 += kMaxLayersPerLaunch;
    } while (l0 < copied);
    if (out_row) *out_row = row;
    return RIC_OK;
}

int32_t ric_compact_plan(const int32_t* refs, int32_t num_blocks, int32_t null_block, int32_t* src, int32_t* dst) {
    if (!refs || num_blocks < 0) return RIC_EINVAL;
    int32_t lo = 0, hi = num_blocks - 1, k = 0;
    for (;;) {
        while (lo < num_blocks && (refs[lo] > 0 || lo == null_block)) ++lo;     // next free page from the bottom
        while (hi >= 0 && (refs[hi] <= 0 || hi == null_block)) --hi;             // next used page from the top
        if (lo >= num_blocks || hi < 0 || lo >= hi) break;
        if (dst) dst[k] = lo;
        if (src) src[k] = hi;
        ++k;
        ++lo;
        --hi;
    }
    return k;
}

}  // extern "C"
