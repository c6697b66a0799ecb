// Log probabilities of given tokens, their rank, the row's entropy and the top
// alternatives.  With m = max x, S = sum e^(x-m) and W = sum e^(x-m) (x-m):
//     logprob = x_t - m - ln S,   entropy = ln S - W / S
// (both terms of the entropy are >= 0, so nothing cancels).  Sums are float32.
//
// Tokens are ordered by (logit descending, id ascending), which a 64-bit key
// holds: the logit's bits mapped to an increasing unsigned number above the
// complement of the id.  -0 counts as +0, a NaN lies above everything.
#include <algorithm>

#include "ric_internal.h"

namespace ric {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float load_logit(const uint8_t* row, int dtype, int64_t i) {
    if (dtype == 2) return reinterpret_cast<const float*>(row)[i];
    const uint16_t h = reinterpret_cast<const uint16_t*>(row)[i];
    if (dtype == 1) return __uint_as_float((uint32_t)h << 16);
    return (float)__builtin_bit_cast(_Float16, h);
}

__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

}  // namespace

// One workgroup per row, the row read once per output it takes (simple form).
__global__ __launch_bounds__(256) void logprobs_simple_kernel(LogprobParams p) {
    __shared__ float fs[4];
    __shared__ unsigned long long ks[4];
    __shared__ int cs[4];
    const int r = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int count = p.dev_count != nullptr ? min(p.max_rows, *p.dev_count) : p.max_rows;
    if (r >= count) return;
    const uint8_t* row = p.logits + (int64_t)r * p.row_stride;
    auto block_sum = [&](float x) {
        for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
        if (lane == 0) fs[w] = x;
        __syncthreads();
        const float t = (fs[0] + fs[1]) + (fs[2] + fs[3]);
        __syncthreads();
        return t;
    };
    auto block_key = [&](unsigned long long k) {
        for (int o = 32; o > 0; o >>= 1) k = max(k, (unsigned long long)__shfl_xor(k, o));
        if (lane == 0) ks[w] = k;
        __syncthreads();
        const unsigned long long t = max(max(ks[0], ks[1]), max(ks[2], ks[3]));
        __syncthreads();
        return t;
    };
    const int target = p.targets != nullptr ? p.targets[r] : -1;
    const bool has = target >= 0 && target < p.vocab;
    const float xt = has ? load_logit(row, p.dtype, target) : 0.f;
    const unsigned long long kt = has ? ((unsigned long long)ordered(xt) << 32) | (uint32_t)~target : 0;
    unsigned long long best = 0;
    int above = 0;
    for (int i = threadIdx.x; i < p.vocab; i += 256) {
        const unsigned long long k = ((unsigned long long)ordered(load_logit(row, p.dtype, i)) << 32) | (uint32_t)~i;
        best = max(best, k);
        above += has && k > kt;
    }
    best = block_key(best);
    const float m = load_logit(row, p.dtype, (int)~(uint32_t)best);
    const bool none = m == -INFINITY;
    float S = 0.f, W = 0.f;
    for (int i = threadIdx.x; i < p.vocab; i += 256) {
        // 0 * -inf has no place in W: below -256 the weight is 0 already
        const float d = fmaxf(load_logit(row, p.dtype, i) - m, -256.f), e = __builtin_amdgcn_exp2f(d * kLog2e);
        S += e;
        W += e * d;
    }
    S = block_sum(S);
    W = block_sum(W);
    for (int o = 32; o > 0; o >>= 1) above += __shfl_xor(above, o);
    if (lane == 0) cs[w] = above;
    __syncthreads();
    const float lnS = __builtin_amdgcn_logf(S) * kLn2;
    auto logp = [&](float x) { return none ? -INFINITY : (x - m) - lnS; };
    if (threadIdx.x == 0) {
        if (p.targets != nullptr) {
            p.logprob[r] = has ? logp(xt) : 0.f;
            p.rank[r] = has ? 1 + cs[0] + cs[1] + cs[2] + cs[3] : 0;
            if (target >= p.vocab && p.status != nullptr) atomicAdd(p.status, 1);
        }
        if (p.entropy != nullptr) p.entropy[r] = none ? 0.f : lnS - W / S;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < p.top_k; ++k) {
        unsigned long long b = 0;
        for (int i = threadIdx.x; i < p.vocab; i += 256) {
            const unsigned long long c = ((unsigned long long)ordered(load_logit(row, p.dtype, i)) << 32) | (uint32_t)~i;
            if (c < last) b = max(b, c);
        }
        last = block_key(b);
        if (threadIdx.x == 0) {
            const int id = (int)~(uint32_t)last;
            p.top_ids[(int64_t)r * p.top_k + k] = id;
            p.top_logprobs[(int64_t)r * p.top_k + k] = logp(load_logit(row, p.dtype, id));
        }
    }
}

size_t logprobs_workspace(int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_logprobs(const LogprobParams& p, void*, hipStream_t s) {
    hipLaunchKernelGGL(logprobs_simple_kernel, dim3(p.max_rows), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace ric
