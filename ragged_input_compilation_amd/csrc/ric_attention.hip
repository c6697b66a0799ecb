// Attention of a step's query tokens over the paged K/V cache.
//
// For query token t of request i at position p, head h, with K/V head h / G:
//     s_j = scale * q.k_j;  s_j = c * tanh(s_j / c) if capped;  s_j -= slope * |p - j|
//     out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// over the keys j < seq_len that are visible: (j <= p or j < prefix) and j > p -
// window.  One pass over the keys with the running maximum m and sum l of the
// softmax; every statistic and accumulator is float32.
#include <algorithm>

#include "ric_internal.h"

namespace ric {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float from_bits16(uint32_t h, bool bf16) {
    if (bf16) return __uint_as_float(h << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// Rounded to nearest even; a NaN stays one.
__device__ __forceinline__ uint16_t to_bits16(float x, bool bf16) {
    if (bf16) return __builtin_bit_cast(uint16_t, (__bf16)x);
    return __builtin_bit_cast(uint16_t, (_Float16)x);
}

// 2^(x log2 e) and tanh of float32: errors of a few units in the last place,
// far below the 8 or 11 bits of the outputs.
__device__ __forceinline__ float tanh_f32(float x) {
    const float e = __builtin_amdgcn_exp2f(x * (2.f * kLog2e));
    return 1.f - 2.f * __builtin_amdgcn_rcpf(e + 1.f);
}

// The request that owns token t (qsl[i] <= t < qsl[i + 1]), or -1: the last i
// with qsl[i] <= t, found by bisection.
__device__ __forceinline__ int request_of(const int32_t* qsl, int n, int t) {
    if (t < qsl[0] || t >= qsl[n]) return -1;
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (qsl[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void raise(int32_t* status) {
    if (status != nullptr) atomicAdd(status, 1);
}

}  // namespace

// ---------------------------------------------------------------------------
// Any head size: one wave per (token, head).  A lane scores one key of a group
// of 64 (its K row in 16-byte pieces against the query in LDS), then the wave
// adds the group's V rows, each lane holding up to four output columns.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void attention_any_kernel(AttnParams p) {
    __shared__ float qs[4][256];
    __shared__ float ps[4][64];
    __shared__ int64_t rows[4][64];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x, h = blockIdx.y * 4 + w;
    if (h >= p.heads) return;
    const int i = request_of(p.qsl, p.num_reqs, t);
    if (i < 0) return;
    const int first = p.qsl[i], n = p.qsl[i + 1] - first, seq = p.seq[i];
    if (n > p.max_q) {
        if (lane == 0 && t == first) raise(p.status);
        return;
    }
    const int pos = seq - n + (t - first);
    const int pre = p.prefix != nullptr ? p.prefix[i] : 0;
    const int end = min(seq, max(pos + 1, pre));
    const int begin = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
    const float slope = p.slopes != nullptr ? p.slopes[h] : 0.f;
    const int kvh = h / (p.heads / p.kv_heads);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q + (int64_t)t * p.q_stride) + (int64_t)h * p.dim;
    for (int d = lane; d < p.dim; d += 64) qs[w][d] = from_bits16(q[d], p.bf16);
    const int64_t row_bytes = (int64_t)p.kv_heads * p.dim * 2;
    const int32_t* table = p.table + (int64_t)i * p.table_stride;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = begin; j0 < end; j0 += 64) {
        const int j = j0 + lane;
        float s = -INFINITY;
        bool bad = false;
        int64_t at = -1;
        if (j < end) {
            const int b = p.block_shift >= 0 ? j >> p.block_shift : j / p.block_size;
            const int64_t id = b < p.table_width ? table[b] : -1;
            if (id < 0 || id >= p.num_blocks) {
                bad = true;
            } else {
                at = (id * p.block_size + (j - b * p.block_size)) * row_bytes + (int64_t)kvh * p.dim * 2;
                float dot = 0.f;
                for (int d = 0; d < p.dim; d += 8) {
                    const u32x4 k = *reinterpret_cast<const u32x4*>(p.kc + at + d * 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dot = fmaf(from_bits16(k[e] & 0xffffu, p.bf16), qs[w][d + 2 * e], dot);
                        dot = fmaf(from_bits16(k[e] >> 16, p.bf16), qs[w][d + 2 * e + 1], dot);
                    }
                }
                s = dot * p.scale;
                if (p.cap > 0.f) s = p.cap * tanh_f32(s / p.cap);
                s -= slope * fabsf((float)(pos - j));
            }
        }
        if (__ballot(bad) != 0 && lane == 0) raise(p.status);
        float top = s;
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        const float m_new = fmaxf(m, top);
        const float base = m_new == -INFINITY ? 0.f : m_new;     // nothing seen yet: every weight is exp(-inf)
        const float keep = __builtin_amdgcn_exp2f((m - base) * kLog2e);
        const float e = at >= 0 ? __builtin_amdgcn_exp2f((s - base) * kLog2e) : 0.f;
        float sum = e;
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
        l = l * keep + sum;
        m = m_new;
        ps[w][lane] = e;
        rows[w][lane] = at;
        __builtin_amdgcn_wave_barrier();
        for (int c = 0; c < 4; ++c) acc[c] *= keep;
        const int cnt = min(64, end - j0);
        for (int k = 0; k < cnt; ++k) {
            if (rows[w][k] < 0) continue;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(p.vc + rows[w][k]);
            const float wgt = ps[w][k];
            for (int c = 0; c < 4; ++c)
                if (c * 64 + lane < p.dim) acc[c] = fmaf(wgt, from_bits16(v[c * 64 + lane], p.bf16), acc[c]);
        }
        __builtin_amdgcn_wave_barrier();
    }
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out + (int64_t)t * p.out_stride) + (int64_t)h * p.dim;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int c = 0; c < 4; ++c)
        if (c * 64 + lane < p.dim) o[c * 64 + lane] = to_bits16(l == 0.f ? 0.f : acc[c] * inv, p.bf16);
}

size_t attention_workspace(const AttnParams&) { return 0; }

hipError_t launch_attention(const AttnParams& p, void*, hipStream_t s) {
    hipLaunchKernelGGL(attention_any_kernel, dim3(p.num_tokens, (p.heads + 3) / 4), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace ric
