// Attention of a step's query tokens over the paged K/V cache.
//
// For query token t of request i at position p, head h, with K/V head h / G:
//     s_j = scale * q.k_j;  s_j = c * tanh(s_j / c) if capped;  s_j -= slope * |p - j|
//     out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// over the keys j < seq_len that are visible: (j <= p or j < prefix) and j > p -
// window.  One pass over the keys with the running maximum m and sum l of the
// softmax; every statistic and accumulator is float32.
#include <algorithm>
#include <type_traits>

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

// Eight 16-bit values as one matrix operand, of either type.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ u32x4 round8(f32x8 x) {
    if constexpr (BF16) return __builtin_bit_cast(u32x4, __builtin_convertvector(x, bf16x8));
    else return __builtin_bit_cast(u32x4, __builtin_convertvector(x, f16x8));
}

// Any 16-bit value of the four words that is infinite or NaN (exponent all ones).
template <bool BF16>
__device__ __forceinline__ bool non_finite(u32x4 x) {
    constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= (x[k] & e) == e || ((x[k] >> 16) & e) == e;
    return bad;
}

// Four 16-bit elements of one column from four consecutive rows: among each 16
// lanes, lane t names 8 bytes of row t / 4 (columns 4 (t % 4)..+3) and receives
// column t of the four rows.
__device__ __forceinline__ uint2 read_transposed(const uint8_t* lds) {
    typedef s16x4 __attribute__((address_space(3)))* lds_ptr;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds)));
}

// Reductions across the four 16-lane groups of a wave, result in every lane.
__device__ __forceinline__ float max_across16(float x) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_across16(float x) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The lowest n bits, n of any value.
__device__ __forceinline__ uint32_t below(int n) {
    return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

// A request as the matrix kernels see it: n query tokens from token `first`, the
// keys [begin, end) that any of its rows can see (begin rounded down to a
// tile), cut into `splits` pieces of `len` keys.
struct Span {
    int first, n, seq, pre, begin, end, splits, len;
};

constexpr int kKeyTile = 32;      // keys per step of a wave

__device__ __forceinline__ Span span_of(const AttnParams& p, int i, int max_splits, int min_len, int tile) {
    Span s;
    s.first = p.qsl[i];
    s.n = p.qsl[i + 1] - s.first;
    if (s.first < 0 || s.n < 0 || s.n > p.num_tokens - s.first) s.n = 0;
    s.seq = p.seq[i];
    s.pre = p.prefix != nullptr ? p.prefix[i] : 0;
    s.end = max(s.seq, 0);
    s.begin = p.window > 0 ? max(0, s.seq - s.n + 1 - p.window) / tile * tile : 0;
    s.begin = min(s.begin, s.end);
    const int keys = s.end - s.begin;
    s.len = max(min_len, ((keys + max_splits - 1) / max_splits + tile - 1) / tile * tile);
    s.splits = max(1, (keys + s.len - 1) / s.len);
    return s;
}

// Pieces of one row's softmax: the unnormalised output, its maximum (in units of
// log2) and sum.
struct Partial {
    float* o;        // [row][split][DP]
    float2* ml;      // [row][split]
};

}  // namespace

// ---------------------------------------------------------------------------
// Few query rows (n tokens x G heads <= 16 NB rows per K/V head): single tokens
// and short drafts.  Bound by reading K and V once.
//
// One workgroup per (request, split of the keys, K/V head); each of its four
// waves takes every fourth tile of 32 keys on its own, no barrier in the loop.
//   S^T = K Q^T: K goes from memory straight into the matrix operand (a lane
//     holds 8 consecutive elements of one key), 16 x 16 x 32 tiles.  A lane's
//     column of S^T is one query row, so softmax statistics are per lane and
//     one exchange across the four 16-lane groups.
//   O^T = V^T P^T: the keys of a tile may be summed in any order, so the S^T
//     registers, rounded to the type, are the P^T operand as they are; V passes
//     through the wave's own piece of LDS and is read back transposed.
// The next tile's K and V are requested as soon as this tile's registers are
// free and its page ids one tile earlier, so 16 KiB per wave are in flight
// through the softmax and the second product.
// P is rounded to the inputs' 8 or 11 bits (the matrix operand's type); its sum
// is taken before the rounding, in float32.
// ---------------------------------------------------------------------------
template <int DP, int NB, bool BF16, bool EXACT>
__global__ __launch_bounds__(256) void attention_rows_kernel(AttnParams p, Partial part, int row_limit, int max_rows,
                                                             int max_splits, int min_len) {
    constexpr int DC = DP / 32;                  // matrix steps along the head
    constexpr int CPR = DP / 8;                  // 16-byte pieces per row
    constexpr int WAVE_LDS = (kKeyTile * DP * 2 > 16 * (DP + 4) * 4) ? kKeyTile * DP * 2 : 16 * (DP + 4) * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[4 * WAVE_LDS];
    __shared__ float2 stats[4][16 * NB];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c16 = lane & 15;
    const int i = blockIdx.x / max_splits, split = blockIdx.x - i * max_splits, kvh = blockIdx.y;
    const int G = p.heads / p.kv_heads;
    const Span sp = span_of(p, i, max_splits, min_len, kKeyTile);
    if (sp.n == 0 || split >= sp.splits) return;
    if (sp.n > p.max_q) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) raise(p.status);
        return;
    }
    const int rows = sp.n * G;
    if (rows > row_limit) return;                // the chunk kernel's
    const int dim = EXACT ? DP : p.dim;
    const int64_t row_bytes = (int64_t)p.kv_heads * dim * 2;
    const int begin = sp.begin + split * sp.len, end = min(sp.end, begin + sp.len);
    const int32_t* table = p.table + (int64_t)i * p.table_stride;
    const uint8_t* kbase = p.kc + (int64_t)kvh * dim * 2 + g * 16;
    const uint8_t* vbase = p.vc + (int64_t)kvh * dim * 2 + g * 16;
    uint8_t* my = lds + w * WAVE_LDS;

    // the query rows (token r / G, head r % G), and their positions and slopes
    u32x4 q[NB][DC];
    int pos[NB];
    float slope[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int r = b * 16 + c16, tok = r / G, h = kvh * G + (r - tok * G);
        const bool in = r < rows;
        const uint8_t* src = p.q + (int64_t)(sp.first + (in ? tok : 0)) * p.q_stride + (int64_t)h * dim * 2 + g * 16;
#pragma unroll
        for (int c = 0; c < DC; ++c) {
            q[b][c] = u32x4{0, 0, 0, 0};
            if (in && (EXACT || c * 32 + g * 8 < dim)) q[b][c] = *reinterpret_cast<const u32x4*>(src + c * 64);
        }
        pos[b] = sp.seq - sp.n + (in ? tok : 0);
        slope[b] = (p.slopes != nullptr && in) ? p.slopes[h] * kLog2e : 0.f;
    }

    f32x4 acc[NB][DP / 16];
    float m[NB], l[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        m[b] = -INFINITY;
        l[b] = 0.f;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) acc[b][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // page id of the lane's two keys (16 s + c16) of a tile; -1 names nothing
    auto page_of = [&](int j) -> int {
        const int blk = p.block_shift >= 0 ? j >> p.block_shift : j / p.block_size;
        return j < end && blk < p.table_width ? table[blk] : -1;
    };
    // A tile's K and V, requested without branches: a key without a page reads
    // the cache's first row instead, and is masked (K) or cleared (V) later.
    u32x4 kr[2][DC], vr[2][DC];
    auto load_tile = [&](int j0, int id0, int id1) -> uint32_t {
        uint64_t has[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int j = j0 + 16 * s + c16, id = s == 0 ? id0 : id1;
            const int blk = p.block_shift >= 0 ? j >> p.block_shift : j / p.block_size;
            const bool ok = (uint32_t)id < (uint64_t)p.num_blocks;
            const int64_t off = ok ? ((int64_t)id * p.block_size + (j - blk * p.block_size)) * row_bytes : 0;
            has[s] = __ballot(ok);
#pragma unroll
            for (int c = 0; c < DC; ++c) {
                const int64_t at_piece = EXACT || c * 32 + g * 8 < dim ? off + c * 64 : off - g * 16;
                kr[s][c] = *reinterpret_cast<const u32x4*>(kbase + at_piece);
                vr[s][c] = *reinterpret_cast<const u32x4*>(vbase + at_piece);
            }
        }
        return (uint32_t)(has[0] & 0xffff) | (uint32_t)(has[1] & 0xffff) << 16;
    };
    // 16-byte piece c of row r in LDS; the pieces of neighbouring rows are turned
    // against each other, so that a column of 16 rows touches every bank
    auto at = [&](int r, int c) { return (r * CPR + (c ^ ((DP == 64 ? r >> 1 : r) & (CPR < 16 ? 7 : 15)))) * 16; };

    const int ntiles = (end - begin + kKeyTile - 1) / kKeyTile;
    int t = w;
    uint32_t have = 0;
    int next0 = -1, next1 = -1;
    if (t < ntiles) {
        const int j = begin + t * kKeyTile + c16;
        const int id0 = page_of(j), id1 = page_of(j + 16);
        next0 = page_of(j + 4 * kKeyTile);
        next1 = page_of(j + 4 * kKeyTile + 16);
        have = load_tile(j - c16, id0, id1);
    }
    bool bad_page = false;
    for (; t < ntiles; t += 4) {
        const int j0 = begin + t * kKeyTile;
        f32x4 sc[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                sc[b][s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < DC; ++c) {
                    const uint32_t in = EXACT || c * 32 + g * 8 < dim ? ~0u : 0u;     // 0 past the head, not NaN
                    sc[b][s] = mfma16<BF16>(kr[s][c] & in, q[b][c], sc[b][s]);
                }
            }
        const uint32_t mask = have;
        if (mask != ~0u) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t keep = (mask >> (16 * s + c16) & 1) ? ~0u : 0u;
#pragma unroll
                for (int c = 0; c < DC; ++c) vr[s][c] &= keep;
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < DC; ++c)
                if (EXACT || c * 32 + g * 8 < dim) *reinterpret_cast<u32x4*>(my + at(16 * s + c16, c * 4 + g)) = vr[s][c];
        const uint32_t inside = end - j0 >= 32 ? ~0u : (1u << (end - j0)) - 1u;
        bad_page |= (mask & inside) != inside;
        // Every row sees every key of the tile, unless the tile lies past the
        // first row's position, behind the last row's window, or has a gap.
        const bool clear = mask == ~0u && j0 + kKeyTile <= max(sp.seq - sp.n + 1, sp.pre) &&
                           (p.window == 0 || j0 > sp.seq - 1 - p.window);
        uint64_t odd_keys[2] = {0, 0};
        if (!clear) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                bool odd = false;                // a non-finite element in the lane's pieces of V
#pragma unroll
                for (int c = 0; c < DC; ++c) odd |= (EXACT || c * 32 + g * 8 < dim) && non_finite<BF16>(vr[s][c]);
                odd_keys[s] = __ballot(odd);
            }
        }
        if (t + 4 < ntiles) {
            have = load_tile(j0 + 4 * kKeyTile, next0, next1);
            next0 = page_of(j0 + 8 * kKeyTile + c16);
            next1 = page_of(j0 + 8 * kKeyTile + c16 + 16);
        }
        u32x4 pr[NB];
        uint32_t sees[NB];                        // the lane's row sees its key 16 s + 4 g + e: bit 16 s + e
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float x[8];
            sees[b] = ~0u;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = sc[b][s][e] * p.scale;
                    if (p.cap > 0.f) v = p.cap * tanh_f32(v / p.cap);
                    x[4 * s + e] = v * kLog2e;
                }
            if (p.slopes != nullptr) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] -= slope[b] * fabsf((float)(pos[b] - (j0 + 16 * (e >> 2) + 4 * g + (e & 3))));
            }
            if (!clear) {
                // keys [lo, hi) of the tile, less those without a page; selected
                // without branches
                const int hi = max(pos[b] + 1, sp.pre) - j0, lo = p.window > 0 ? pos[b] - p.window + 1 - j0 : 0;
                sees[b] = (mask & below(hi) & ~below(lo)) >> (4 * g);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = (sees[b] >> (16 * (e >> 2) + (e & 3)) & 1) ? x[e] : -INFINITY;
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
            top = fmaxf(m[b], max_across16(top));
            const float base = top == -INFINITY ? 0.f : top;
            const float keep = __builtin_amdgcn_exp2f(m[b] - base);
            m[b] = top;
            float sum = 0.f;
            f32x8 pe;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                pe[e] = __builtin_amdgcn_exp2f(x[e] - base);
                sum += pe[e];
            }
            l[b] = l[b] * keep + sum;            // the lane's own keys; the groups are added at the end
            pr[b] = round8<BF16>(pe);
            if (__ballot(keep != 1.f) != 0) {
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) acc[b][d] *= keep;
            }
        }
        const uint32_t odd_tile = (uint32_t)(((odd_keys[0] | odd_keys[0] >> 16 | odd_keys[0] >> 32 | odd_keys[0] >> 48) & 0xffff) |
                                             ((odd_keys[1] | odd_keys[1] >> 16 | odd_keys[1] >> 32 | odd_keys[1] >> 48) & 0xffff) << 16);
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
            if (!EXACT && d * 16 >= dim) continue;
            uint2 half[2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
                half[s] = read_transposed(my + at(16 * s + 4 * g + (c16 >> 2), 2 * d + ((c16 & 3) >> 1)) + (c16 & 1) * 8);
            const u32x4 vt = {half[0].x, half[0].y, half[1].x, half[1].y};
            if (odd_tile == 0) {
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[b][d] = mfma16<BF16>(vt, pr[b], acc[b][d]);
            } else {
                // A masked tile with infinities or NaN among its values: 0 times
                // them would reach rows that do not see them.  The finite keys go
                // together; each of the others alone, added only where it is seen.
                for (uint32_t todo = odd_tile, step = 0; step == 0 || todo != 0; ++step) {
                    const uint32_t one = step == 0 ? 0u : todo & (0u - todo);
                    if (step > 0) todo &= todo - 1;
                    const uint32_t keys = step == 0 ? ~odd_tile : one;
                    // the lane's eight keys, as masks of the four words
                    const uint32_t lo4 = keys >> (4 * g), hi4 = keys >> (16 + 4 * g);
                    auto pair = [](uint32_t two) { return ((two & 1) ? 0xffffu : 0u) | ((two & 2) ? 0xffff0000u : 0u); };
                    const u32x4 part_v = vt & u32x4{pair(lo4), pair(lo4 >> 2), pair(hi4), pair(hi4 >> 2)};
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const f32x4 add = mfma16<BF16>(part_v, pr[b], f32x4{0.f, 0.f, 0.f, 0.f});
                        // does the lane's row see the key?  its group holds the answer
                        const int key = __ffs(one) - 1;
                        const int holder = (key >> 2 & 3) * 16 + c16, bit = (key & 16) + (key & 3);
                        const bool see = step == 0 || (__shfl((int)sees[b], step == 0 ? lane : holder) >> (step == 0 ? 0 : bit) & 1);
                        if (see) acc[b][d] += add;
                    }
                }
            }
        }
    }
    if (bad_page && lane == 0) raise(p.status);

    // The four waves' pieces: common maximum, scaled sums, added through LDS.
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        l[b] = sum_across16(l[b]);
        if (g == 0) stats[w][b * 16 + c16] = make_float2(m[b], l[b]);
    }
    __syncthreads();
    const int row16 = threadIdx.x >> 4, piece = threadIdx.x & 15;       // 16 threads per row
    constexpr int DT = DP / 16;                                         // outputs per thread
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float top = -INFINITY;
        for (int k = 0; k < 4; ++k) top = fmaxf(top, stats[k][b * 16 + c16].x);
        const float f = m[b] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[b] - top);
        float* mine = reinterpret_cast<float*>(my);
        if (b > 0) __syncthreads();
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
            *reinterpret_cast<f32x4*>(mine + c16 * (DP + 4) + d * 16 + 4 * g) =
                m[b] == -INFINITY ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[b][d] * f;
        __syncthreads();
        const int r = b * 16 + row16;
        if (r < rows) {
            float rt = -INFINITY, rl = 0.f;
            for (int k = 0; k < 4; ++k) rt = fmaxf(rt, stats[k][r].x);
            for (int k = 0; k < 4; ++k)
                // no maximum: the sum is 0, or NaN where every score was
                rl += stats[k][r].x == -INFINITY ? stats[k][r].y : stats[k][r].y * __builtin_amdgcn_exp2f(stats[k][r].x - rt);
            float o[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                o[d] = 0.f;
                for (int k = 0; k < 4; ++k)
                    o[d] += reinterpret_cast<const float*>(lds + k * WAVE_LDS)[row16 * (DP + 4) + piece * DT + d];
            }
            const int tok = r / G, h = kvh * G + (r - tok * G);
            if (sp.splits == 1) {
                const float inv = rl == 0.f ? 0.f : 1.f / rl;
                uint16_t* dst = reinterpret_cast<uint16_t*>(p.out + (int64_t)(sp.first + tok) * p.out_stride) + (int64_t)h * dim;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    if (EXACT || piece * DT + d < dim) dst[piece * DT + d] = to_bits16(rl == 0.f ? 0.f : o[d] * inv, BF16);
            } else {
                const int64_t at_row = (((int64_t)i * p.kv_heads + kvh) * max_rows + r) * max_splits + split;
#pragma unroll
                for (int d = 0; d < DT; ++d) part.o[at_row * DP + piece * DT + d] = o[d];
                if (piece == 0) part.ml[at_row] = make_float2(rt, rl);
            }
        }
    }
}

// Joins the splits of one row: one workgroup per (request, row of a K/V head),
// DP / 4 threads per split, the splits in a fixed order.
template <int DP>
__global__ __launch_bounds__(256) void join_rows_kernel(AttnParams p, Partial part, int row_limit, int max_rows,
                                                        int max_splits, int min_len) {
    constexpr int T = DP / 4, S = 256 / T;       // threads per split, splits at a time
    __shared__ f32x4 sums[S][T];
    __shared__ float lsum[S];
    const int i = blockIdx.x, kvh = blockIdx.y / max_rows, r = blockIdx.y - kvh * max_rows;
    const int G = p.heads / p.kv_heads;
    const Span sp = span_of(p, i, max_splits, min_len, kKeyTile);
    if (sp.n == 0 || sp.n > p.max_q || sp.n * G > row_limit || sp.splits == 1 || r >= sp.n * G) return;
    const int64_t row = (((int64_t)i * p.kv_heads + kvh) * max_rows + r) * max_splits;
    float top = -INFINITY;
    for (int s = threadIdx.x & 63; s < sp.splits; s += 64) top = fmaxf(top, part.ml[row + s].x);
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const int d4 = threadIdx.x % T, sub = threadIdx.x / T;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll 4
    for (int s = sub; s < sp.splits; s += S) {
        const float2 ml = part.ml[row + s];
        const float f = ml.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
        const f32x4 v = *reinterpret_cast<const f32x4*>(part.o + (row + s) * DP + d4 * 4);
        if (ml.x != -INFINITY) o += v * f;
        l += ml.x == -INFINITY ? ml.y : ml.y * f;      // no maximum: 0, or NaN where every score was
    }
    sums[sub][d4] = o;
    if (d4 == 0) lsum[sub] = l;
    __syncthreads();
    if (sub != 0 || d4 * 4 >= p.dim) return;
    for (int k = 1; k < S; ++k) {
        o += sums[k][d4];
        l += lsum[k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = r / G, h = kvh * G + (r - tok * G);
    uint16_t* dst = reinterpret_cast<uint16_t*>(p.out + (int64_t)(sp.first + tok) * p.out_stride) + (int64_t)h * p.dim + d4 * 4;
    for (int e = 0; e < 4; ++e) dst[e] = to_bits16(l == 0.f ? 0.f : o[e] * inv, p.bf16);
}

// ---------------------------------------------------------------------------
// Any head size: one wave per (token, head).  A lane scores one key of a group
// of 64 (its K row in 16-byte pieces against the query in LDS), then the wave
// adds the group's V rows, each lane holding up to four output columns.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void attention_any_kernel(AttnParams p, int row_limit) {
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
    if (n * (p.heads / p.kv_heads) <= row_limit) return;
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

namespace {

// How a call is cut: by what the host knows, and for every length that the
// device may hold.
struct Plan {
    int nb;              // 16-row blocks of the few-rows kernel, 0: not launched
    int row_limit;       // its largest request, in rows per K/V head
    int max_rows;        // rows its partial results are laid out for
    int splits;          // most pieces of a request's keys
    int min_len;         // fewest keys per piece
    bool chunks;         // some request may be larger
    int dp;              // head size of the kernels
};

constexpr int kTargetGroups = 2048;      // workgroups that keep 256 CUs evenly busy
constexpr int kMinSplitLen = 256;

Plan plan_of(const AttnParams& p) {
    Plan r{};
    const int G = p.heads / p.kv_heads;
    const int64_t most = (int64_t)p.max_q * G;
    r.dp = p.dim <= 64 ? 64 : p.dim <= 128 ? 128 : 256;
    if (most <= 64) {
        r.nb = most <= 16 ? 1 : most <= 32 ? 2 : 4;
    } else if (G <= 64) {
        r.nb = G <= 16 ? 1 : G <= 32 ? 2 : 4;
        r.chunks = true;
    } else {
        r.chunks = true;
    }
    r.row_limit = 16 * r.nb;
    r.max_rows = (int)std::min<int64_t>(most, r.row_limit);
    const int64_t keys = p.window > 0 && p.prefix == nullptr ? std::min<int64_t>(p.max_seq, (int64_t)p.window + p.max_q + 31) : p.max_seq;
    const int64_t groups = std::max<int64_t>(1, (int64_t)p.num_reqs * p.kv_heads);
    const int64_t want = std::max<int64_t>(1, kTargetGroups / groups);
    r.min_len = (int)std::max<int64_t>(kMinSplitLen, ((keys + want - 1) / want + 31) / 32 * 32);
    r.min_len = std::min(r.min_len, 1024);
    r.splits = (int)std::max<int64_t>(1, std::min<int64_t>((keys + r.min_len - 1) / r.min_len, 256));
    return r;
}

int64_t partial_rows(const AttnParams& p, const Plan& r) {
    return r.splits > 1 ? (int64_t)p.num_reqs * p.kv_heads * r.max_rows * r.splits : 0;
}

template <int DP, bool BF16, bool EXACT>
void launch_rows(const AttnParams& p, const Plan& r, Partial part, hipStream_t s) {
    const dim3 grid((uint32_t)(p.num_reqs * r.splits), p.kv_heads);
    if (r.nb == 1)
        hipLaunchKernelGGL((attention_rows_kernel<DP, 1, BF16, EXACT>), grid, dim3(256), 0, s, p, part, r.row_limit, r.max_rows, r.splits, r.min_len);
    else if (r.nb == 2)
        hipLaunchKernelGGL((attention_rows_kernel<DP, 2, BF16, EXACT>), grid, dim3(256), 0, s, p, part, r.row_limit, r.max_rows, r.splits, r.min_len);
    else
        hipLaunchKernelGGL((attention_rows_kernel<DP, 4, BF16, EXACT>), grid, dim3(256), 0, s, p, part, r.row_limit, r.max_rows, r.splits, r.min_len);
    if (r.splits > 1)
        hipLaunchKernelGGL((join_rows_kernel<DP>), dim3(p.num_reqs, p.kv_heads * r.max_rows), dim3(256), 0, s, p, part, r.row_limit, r.max_rows, r.splits, r.min_len);
}

}  // namespace

size_t attention_workspace(const AttnParams& p) {
    const Plan r = plan_of(p);
    return (size_t)partial_rows(p, r) * (r.dp * 4 + 8);
}

hipError_t launch_attention(const AttnParams& p, void* workspace, hipStream_t s) {
    const Plan r = plan_of(p);
    Partial part{};
    part.o = static_cast<float*>(workspace);
    part.ml = reinterpret_cast<float2*>(part.o + partial_rows(p, r) * r.dp);
    if (r.nb > 0) {
        auto go = [&](auto dp, auto bf16) {
            constexpr int DP = decltype(dp)::value;
            constexpr bool BF = decltype(bf16)::value;
            if (p.dim == DP) launch_rows<DP, BF, true>(p, r, part, s);
            else launch_rows<DP, BF, false>(p, r, part, s);
        };
        auto by_dim = [&](auto bf16) {
            if (r.dp == 64) go(std::integral_constant<int, 64>{}, bf16);
            else if (r.dp == 128) go(std::integral_constant<int, 128>{}, bf16);
            else go(std::integral_constant<int, 256>{}, bf16);
        };
        if (p.bf16) by_dim(std::true_type{}); else by_dim(std::false_type{});
    }
    if (r.chunks)
        hipLaunchKernelGGL(attention_any_kernel, dim3(p.num_tokens, (p.heads + 3) / 4), dim3(256), 0, s, p, r.row_limit);
    return hipGetLastError();
}

}  // namespace ric
