// The handle and the host helpers that more than one source file uses: the
// persistent batch's row maps, counters and staging state (ric_host.cpp), and
// the page calls that work on the same tables (ric_ops_host.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <unordered_map>
#include <vector>

#include "../../include/ric.h"
#include "ric_internal.h"

namespace ric {

// Records the message of the calling thread's failed call; returns `code`.
int fail(int code, const char* fmt, ...);

#define HIP_TRY(expr)                                                                   \
    do {                                                                                \
        hipError_t e_ = (expr);                                                         \
        if (e_ != hipSuccess) return fail(RIC_EHIP, "%s: %s", #expr, hipGetErrorString(e_)); \
    } while (0)

constexpr size_t kAlign = 256;
constexpr int32_t kMaxRowsPerLaunch = 1 << 24;   // rows * 256 lanes must fit a 32-bit work-item count

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int ilog2_exact(int64_t x) {
    if (x <= 0 || (x & (x - 1)) != 0) return -1;
    int s = 0;
    while ((int64_t(1) << s) < x) ++s;
    return s;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Layout {
    int64_t tok_stride, blk_stride;
    size_t off_tok, off_blk, off_scal, off_ids, off_pos, off_req, off_slot, off_qsl, off_seq,
        off_logits, off_sample, off_discard, off_dscal, off_pairs, off_cuk, off_samp_off, off_samp_idx,
        off_spec_logits, off_spec_target, off_spec_draft, off_spec_cu, off_spec_bonus, off_spec_d,
        off_corr, off_pages, off_staging, total;
    size_t staging_bytes;
    // KV-cache groups 1..groups-1 (index g): block tables and slot outputs
    int groups;
    int64_t xblk_stride[kMaxGroups];
    size_t off_xblk[kMaxGroups], off_xslot[kMaxGroups];
};

int num_groups_of(const ric_config& c);
int32_t group_B(const ric_config& c, int g);
int32_t group_pool(const ric_config& c, int g);
int32_t group_cap(const ric_config& c, int g);

}  // namespace ric

struct ric_batch {
    ric_config cfg{};
    ric::Layout L{};
    hipStream_t stream = nullptr;
    int device = 0;
    bool own_ws = false;
    uint8_t* ws = nullptr;

    // device regions
    int32_t *d_tok = nullptr, *d_blk = nullptr, *d_scal = nullptr;
    int32_t* d_xblk[ric::kMaxGroups] = {nullptr, nullptr, nullptr, nullptr};    // groups 1..
    int32_t* d_xslot[ric::kMaxGroups] = {nullptr, nullptr, nullptr, nullptr};
    int32_t *d_ids = nullptr, *d_pos = nullptr, *d_req = nullptr, *d_slot = nullptr;
    int32_t *d_qsl = nullptr, *d_seq = nullptr, *d_logits = nullptr, *d_sample = nullptr;
    uint8_t* d_discard = nullptr;
    int32_t *d_dscal = nullptr, *d_pairs = nullptr, *d_cuk = nullptr, *d_samp_idx = nullptr;
    int64_t* d_samp_off = nullptr;
    int32_t *d_spec_logits = nullptr, *d_spec_target = nullptr, *d_spec_draft = nullptr,
            *d_spec_cu = nullptr, *d_spec_bonus = nullptr, *d_spec_d = nullptr;
    int32_t* d_corr = nullptr;       // [3][max_num_reqs]: rows, sampler positions, draft counts
    int32_t* d_pages = nullptr;      // [kMaxPagePairs][2]: page copies being made
    uint8_t* d_staging = nullptr;

    // pinned delta logs
    uint8_t* h_log[2] = {nullptr, nullptr};
    uint8_t* d_log[2] = {nullptr, nullptr};  // device addresses of the same pinned logs
    hipEvent_t ev[2] = {nullptr, nullptr};
    bool ev_pending[2] = {false, false};
    int cur = 0;
    bool cur_ready = false;          // h_log[cur] is known free to write
    uint32_t payload_words = 0;
    std::vector<ric::DeltaOp> ops;
    uint32_t epoch = 1;

    // host mirror
    std::vector<int32_t> scal;       // [ric::kNumScalarCols][max_num_reqs]
    int32_t dirty_lo[ric::kNumScalarCols], dirty_hi[ric::kNumScalarCols];
    std::vector<uint64_t> req_at;
    std::vector<uint8_t> live;
    std::vector<uint32_t> pending_epoch;
    std::unordered_map<uint64_t, int32_t> row_of;
    int32_t num_live = 0;

    // schedule state
    bool scheduled = false;
    bool compiled = false;           // a compile ran since the last schedule
    bool corrected = false;          // ric_correct_computed ran since the last schedule
    int32_t sched_R = 0, sched_N = 0, sched_max_q = 0, sched_max_seq = 0, sched_sampled = 0;

    int32_t& S(int col, int row) { return scal[(size_t)col * cfg.max_num_reqs + row]; }
    int32_t* dcol(int col) { return d_scal + (size_t)col * cfg.max_num_reqs; }

    void mark(int col, int row) {
        dirty_lo[col] = std::min(dirty_lo[col], row);
        dirty_hi[col] = std::max(dirty_hi[col], row + 1);
    }
    void clear_dirty() {
        for (int c = 0; c < ric::kNumScalarCols; ++c) {
            dirty_lo[c] = cfg.max_num_reqs;
            dirty_hi[c] = 0;
        }
    }
    int32_t used_rows() const {
        for (int32_t r = cfg.max_num_reqs - 1; r >= 0; --r)
            if (live[r]) return r + 1;
        return 0;
    }
    // block table of KV-cache group g
    int32_t* blk(int g) const { return g == 0 ? d_blk : d_xblk[g]; }
    int64_t bstride(int g) const { return g == 0 ? L.blk_stride : L.xblk_stride[g]; }
};

namespace ric {

// Makes the handle's device current for one call (and restores the caller's),
// so a process that drives handles on several GPUs needs no device switching
// of its own around library calls.
struct DeviceScope {
    int prev = -1;
    explicit DeviceScope(const ric_batch* b) {
        int cur = -1;
        if (hipGetDevice(&cur) == hipSuccess && cur != b->device && hipSetDevice(b->device) == hipSuccess) prev = cur;
    }
    ~DeviceScope() {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
    DeviceScope(const DeviceScope&) = delete;
    DeviceScope& operator=(const DeviceScope&) = delete;
};

// Stage `n` words for device address `dst`, splitting across ops and flushes.
int stage(ric_batch* b, void* dst, const void* src, size_t n);
// Upload what is staged.
int flush(ric_batch* b);
// ESTATE while the handle's stream is being captured into a graph.
int refuse_if_capturing(ric_batch* b);
// Flush first when a new whole-row write could overlap a staged write to the
// same row (ops of one flush are applied in parallel).
int before_row_overwrite(ric_batch* b, int32_t row);
// Every id usable: inside group g's pool and not the null block.
int check_blocks(const ric_batch* b, int g, const int32_t* ids, int32_t n);
int find(const ric_batch* b, uint64_t req_id, int32_t* row);
int32_t as_bits(float f);

}  // namespace ric
