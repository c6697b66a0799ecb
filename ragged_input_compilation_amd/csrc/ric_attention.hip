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

// tanh(x) from y = 2 x log2 e: an error of a few 2^-24, far below the 8 or 11 bits
// of the outputs.
__device__ __forceinline__ float tanh_of(float y) {
    return 1.f - 2.f * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(y) + 1.f);
}

// Factors of a call that hold for every score: products q.k come to units of log2
// by `log2`; under a cap by cap * tanh_of(q.k * arg).  Kept finite, so that a
// product of 0 stays 0 under the largest scales.
struct Factors {
    float log2, arg, cap;
    __device__ static float finite(float x) { return fminf(fmaxf(x, -3.4028235e38f), 3.4028235e38f); }
    __device__ explicit Factors(const AttnParams& p)
        : log2(finite(p.scale * kLog2e)), arg(p.cap > 0.f ? finite(p.scale / p.cap * (2.f * kLog2e)) : 0.f),
          cap(finite(p.cap * kLog2e)) {}
};

__device__ __forceinline__ void raise(int32_t* status) {
    if (status != nullptr) atomicAdd(status, 1);
}

// Eight 16-bit values as one matrix operand, of either type.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ u32x4 round8(f32x8 x) {
    if constexpr (BF16) return __builtin_bit_cast(u32x4, __builtin_convertvector(x, bf16x8));
    else return __builtin_bit_cast(u32x4, __builtin_convertvector(x, f16x8));
}

// Four 16-bit elements of one column from four consecutive rows: among each 16
// lanes, lane t names 8 bytes of row t / 4 (columns 4 (t % 4)..+3) and receives
// column t of the four rows.
__device__ __forceinline__ uint2 read_transposed(const __attribute__((address_space(3))) uint8_t* lds) {
    typedef s16x4 __attribute__((address_space(3)))* lds_ptr;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds)));
}

// Set where one of the eight 16-bit values is infinite or NaN (exponent all
// ones: adding its lowest bit carries into the sign's place).
template <bool BF16>
__device__ __forceinline__ uint32_t odd_bits(u32x4 x) {
    constexpr uint32_t e = BF16 ? 0x7f807f80u : 0x7c007c00u, one = BF16 ? 0x00800080u : 0x04000400u;
    uint32_t f = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) f |= (x[k] & e) + one;
    return f & 0x80008000u;
}

// Across the two halves of a wave, result in every lane.
__device__ __forceinline__ float max_across32(float x) {
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_across32(float x) {
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
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
// keys [begin, end) that any of its rows can see and its table can name (begin
// rounded down to a tile), cut into `splits` pieces of `len` keys.
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
    // keys past the table have no page: left out, and reported where seq > end
    s.end = min(max(s.seq, 0), (int)min((int64_t)p.table_width * p.block_size, (int64_t)1 << 30));
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

// How a call's work is cut (see plan_of).
struct Cut {
    int row_limit;   // largest request of the few-rows part, in rows per K/V head
    int max_rows;    // rows its partial results are laid out for
    int splits;      // most pieces of a request's keys
    int min_len;     // fewest keys per piece
    int row_groups;  // workgroups of the few-rows part
    int tile_groups; // workgroups of the many-rows part
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
// Measured (32 heads over 8 of 128, bf16): 256 tokens over up to 4096 keys each 436
// us, 5.14 TB/s; one token over 60001 keys 43 us and 10 for the join, 5.6 TB/s.
// ---------------------------------------------------------------------------
template <int DP>
constexpr int kRowsWaveLds = (kKeyTile * DP * 2 > 16 * (DP + 4) * 4) ? kKeyTile * DP * 2 : 16 * (DP + 4) * 4;
template <int DP, int NB>
constexpr int kRowsLds = 4 * kRowsWaveLds<DP> + 4 * 16 * NB * 8;      // bytes of LDS

template <int DP, int NB, bool BF16, bool EXACT>
__device__ __forceinline__ void rows_group(const AttnParams& p, const Partial& part, const Cut& cut, int group, uint8_t* lds) {
    constexpr int DC = DP / 32;                  // matrix steps along the head
    constexpr int CPR = DP / 8;                  // 16-byte pieces per row
    constexpr int WAVE_LDS = kRowsWaveLds<DP>;
    auto stats = reinterpret_cast<float2 (*)[16 * NB]>(lds + 4 * WAVE_LDS);
    const int row_limit = cut.row_limit, max_rows = cut.max_rows, max_splits = cut.splits, min_len = cut.min_len;
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c16 = lane & 15;
    const int pieces = p.num_reqs * max_splits, kvh = group / pieces, piece_of = group - kvh * pieces;
    const int i = piece_of / max_splits, split = piece_of - i * max_splits;
    const int G = p.heads / p.kv_heads;
    const Span sp = span_of(p, i, max_splits, min_len, kKeyTile);
    if (sp.n == 0 || split >= sp.splits) return;
    if (sp.n > p.max_q) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) raise(p.status);
        return;
    }
    const int rows = sp.n * G;
    if (rows > row_limit) return;                // the chunk kernel's
    if (sp.seq > sp.end && threadIdx.x == 0 && split == 0 && kvh == 0) raise(p.status);
    const int dim = EXACT ? DP : p.dim;
    const int64_t row_bytes = (int64_t)p.kv_heads * dim * 2;
    const int begin = sp.begin + split * sp.len, end = min(sp.end, begin + sp.len);
    const int32_t* table = p.table + (int64_t)i * p.table_stride;
    const uint8_t* kbase = p.kc + (int64_t)kvh * dim * 2 + g * 16;
    const uint8_t* vbase = p.vc + (int64_t)kvh * dim * 2 + g * 16;
    uint8_t* my = lds + w * WAVE_LDS;
    const Factors by(p);

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
                for (int c = 0; c < DC; ++c) odd |= (EXACT || c * 32 + g * 8 < dim) && odd_bits<BF16>(vr[s][c]) != 0;
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
            if (p.cap > 0.f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = by.cap * tanh_of(sc[b][e >> 2][e & 3] * by.arg);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = sc[b][e >> 2][e & 3] * by.log2;
            }
            if (p.slopes != nullptr) {
                const float d = (float)(pos[b] - (j0 + 4 * g));      // exact below 2^24, as all its steps
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] -= slope[b] * fabsf(d - (float)(16 * (e >> 2) + (e & 3)));
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
                half[s] = read_transposed((const __attribute__((address_space(3))) uint8_t*)my + at(16 * s + 4 * g + (c16 >> 2), 2 * d + ((c16 & 3) >> 1)) + (c16 & 1) * 8);
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

template <int DP, int NB, bool BF16, bool EXACT>
__global__ __launch_bounds__(256, NB == 1 ? 2 : 1) void attention_rows_kernel(AttnParams p, Partial part, Cut cut) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[kRowsLds<DP, NB>];
    rows_group<DP, NB, BF16, EXACT>(p, part, cut, blockIdx.x, lds);
}

// Joins the splits of one row: one workgroup per (request, row of a K/V head),
// DP / 4 threads per split, the splits in a fixed order.
template <int DP>
__global__ __launch_bounds__(256) void join_rows_kernel(AttnParams p, Partial part, Cut cut) {
    const int row_limit = cut.row_limit, max_rows = cut.max_rows, max_splits = cut.splits, min_len = cut.min_len;
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
#pragma unroll 8
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

// One row by one wave, key by key where the weights meet V: the way out for rows
// that stand next to infinities or NaN they do not see.  A lane scores one key of
// a group of 64, then the wave adds the group's V rows, each lane holding up to
// four output columns.  `scratch`: 1.75 KiB of LDS of the wave's own.
__device__ __forceinline__ void exact_row(const AttnParams& p, const int32_t* table, int tok, int head, int kvh, int pos, int begin,
                                       int end, uint8_t* scratch) {
    const int lane = threadIdx.x & 63;
    float* qs = reinterpret_cast<float*>(scratch);
    float* ps = qs + 256;
    int64_t* at = reinterpret_cast<int64_t*>(ps + 64);
    const float slope = p.slopes != nullptr ? p.slopes[head] * kLog2e : 0.f;
    const Factors by(p);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q + (int64_t)tok * p.q_stride) + (int64_t)head * p.dim;
    for (int d = lane; d < p.dim; d += 64) qs[d] = from_bits16(q[d], p.bf16);
    const int64_t row_bytes = (int64_t)p.kv_heads * p.dim * 2;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = begin; j0 < end; j0 += 64) {
        const int j = j0 + lane, blk = p.block_shift >= 0 ? j >> p.block_shift : j / p.block_size;
        const int64_t id = j < end && blk < p.table_width ? table[blk] : -1;
        const int64_t where = id >= 0 && id < p.num_blocks
            ? (id * p.block_size + (j - blk * p.block_size)) * row_bytes + (int64_t)kvh * p.dim * 2 : -1;
        float s = -INFINITY;
        if (where >= 0) {
            float dot = 0.f;
            for (int d = 0; d < p.dim; d += 8) {
                const u32x4 k = *reinterpret_cast<const u32x4*>(p.kc + where + d * 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dot = fmaf(from_bits16(k[e] & 0xffffu, p.bf16), qs[d + 2 * e], dot);
                    dot = fmaf(from_bits16(k[e] >> 16, p.bf16), qs[d + 2 * e + 1], dot);
                }
            }
            s = p.cap > 0.f ? by.cap * tanh_of(dot * by.arg) : dot * by.log2;
            s -= slope * fabsf((float)(pos - j));
        }
        float top = s;
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        const float m_new = fmaxf(m, top), base = m_new == -INFINITY ? 0.f : m_new;
        const float keep = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - base);
        const float e = where >= 0 ? __builtin_amdgcn_exp2f(s - base) : 0.f;
        float sum = e;
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
        l = l * keep + sum;
        m = m_new;
        ps[lane] = e;
        at[lane] = where;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] *= keep;
        for (int k = 0; k < min(64, end - j0); ++k) {
            if (at[k] < 0) continue;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(p.vc + at[k]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c * 64 + lane < p.dim) acc[c] = fmaf(ps[k], from_bits16(v[c * 64 + lane], p.bf16), acc[c]);
        }
        __builtin_amdgcn_wave_barrier();
    }
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out + (int64_t)tok * p.out_stride) + (int64_t)head * p.dim;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c * 64 + lane < p.dim) o[c * 64 + lane] = to_bits16(l == 0.f ? 0.f : acc[c] * inv, p.bf16);
}

// ---------------------------------------------------------------------------
// Many query rows (chunks).  Bound by the matrix products and the exponentials
// between them.
//
// The n x G rows of a request's K/V head (row R: token R / G, head R % G, so that
// neighbouring rows share positions and the tile's keys) are cut into tiles of
// 128; a workgroup takes one tile, each of its four waves 32 rows, and walks the
// keys in tiles of KT that all four share through LDS.  Tile x of the grid
// belongs to the last request i with start_i = qsl[i] * G / 128 + i <= x: starts
// that far apart hold every request's tiles, and need no prefix sum.
//   S^T = K Q^T and O^T = V^T P^T on 32 x 32 x 16 products, as in the few-rows
//   kernel: a lane's column is one query row, P^T is S^T rounded in place, V is
//   read back from LDS transposed.  The other 16 keys of a row sit in lane ^ 32.
//   K and V go from memory to LDS without registers (16 bytes per lane, the next
//   tile while this one is computed); the lanes of a load pick which piece of
//   which row they fetch, which turns rows against each other (no bank is hit
//   more often than the access needs).  A key past the end fetches the last one,
//   a key without a page the cache's first row; both are masked.
//   The maximum a row is scaled by is only raised when a new one exceeds it by
//   more than 2^8, so most tiles leave the 64 accumulators untouched.
//   P is summed after its rounding to the type, so that weights and sum agree.
// Measured (32 heads over 8 of 128, bf16): 4 chunks of 2048 over up to 30720 keys
// 1990 us, 1023 TFLOP/s, where an 8192^3 library product reaches 1167.  Two workgroups
// per CU overlap one's products with the other's exponentials; two row blocks per
// wave, a ring of four tiles and three workgroups took 2 to 20% longer.
// ---------------------------------------------------------------------------
constexpr int kRowTile = 128;

template <int DP>
struct ChunkShape {
    static constexpr int KT = DP <= 128 ? 64 : 32;         // keys per tile
    static constexpr int KB = KT / 32;
    static constexpr int CPR = DP / 8;                     // 16-byte pieces per row
    static constexpr int TILE = KT * DP * 2;               // bytes of one K or V tile
    static constexpr int LOADS = TILE / (4 * 1024);        // loads of 1 KiB per wave
    static constexpr int LDS = 4 * TILE + 16;
    // Where piece c of row r lies in its row.  A transposed read takes four
    // neighbouring pieces of eight neighbouring rows, a K read one or two pieces
    // of 32: both spread over all 256 bytes of banks.
    __device__ static int turn(int r) {
        if constexpr (DP == 64) return ((r >> 1 & 1) << 2) | (r >> 2 & 3);
        else return ((r & 3) << 2) | (r >> 2 & 3);
    }
};

// Copies 16 bytes per lane from memory (base + offset) to LDS at `lds` + 16 * lane.
// Complete after s_waitcnt vmcnt(0).  Written as text because the compiler, given
// its own form, waits for the load in flight before every read of the other
// tile.  It writes no vector register; M0, which holds the LDS address, is left
// as it was.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const uint8_t* base, uint32_t offset) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(base) : "memory");
}
// The same from any 64-bit address.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const uint8_t* src) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src) : "memory");
}

// Eight values' sum added to `sum`, from the rounded pairs.
template <bool BF16>
__device__ __forceinline__ float add_pairs(u32x4 x, float sum) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t two = x[k];
        if constexpr (BF16)
            sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), bf16x2{(__bf16)1.f, (__bf16)1.f}, sum, false);
        else
            sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, two), f16x2{(_Float16)1.f, (_Float16)1.f}, sum, false);
    }
    return sum;
}

template <int DP, bool BF16, bool EXACT, bool FEAT>
__device__ __forceinline__ void chunk_group(const AttnParams& p, const Cut& cut, int group, uint8_t* lds) {
    using Shape = ChunkShape<DP>;
    constexpr int KT = Shape::KT, KB = Shape::KB, CPR = Shape::CPR, TILE = Shape::TILE;
    constexpr int QS = DP / 16, DB = DP / 32;
    // [2][K, V] tiles from LDS offset 0 (a load to LDS reaches 64 KiB), then a flag:
    // a page that names nothing was met
    // (an LDS pointer: a flat or volatile read would wait for the loads in flight)
    __attribute__((address_space(3))) int* gap = (__attribute__((address_space(3))) int*)(lds + 4 * TILE);
    const int row_limit = cut.row_limit;
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, h32 = lane >> 5, c32 = lane & 31;
    // neighbouring workgroups (which go to different XCDs) take different K/V
    // heads; the last tiles, with the most keys, go first
    const int kvh = group % p.kv_heads;
    const int x = cut.tile_groups / p.kv_heads - 1 - group / p.kv_heads;
    const int G = p.heads / p.kv_heads;
    auto start = [&](int i) { return (int)((int64_t)p.qsl[i] * G / kRowTile) + i; };
    int i = 0;
    for (int hi = p.num_reqs - 1; i < hi;) {
        const int mid = (i + hi + 1) >> 1;
        if (start(mid) <= x) i = mid; else hi = mid - 1;
    }
    const Span sp = span_of(p, i, 1, 1, 1);
    const int row0 = (x - start(i)) * kRowTile, rows = sp.n * G;
    if (row0 < 0 || row0 >= rows || rows <= row_limit) return;
    if (sp.n > p.max_q) {
        if (threadIdx.x == 0 && row0 == 0 && kvh == 0) raise(p.status);
        return;
    }
    if (sp.seq > sp.end && threadIdx.x == 0 && row0 == 0 && kvh == 0) raise(p.status);
    const int dim = EXACT ? DP : p.dim;
    const int64_t row_bytes = (int64_t)p.kv_heads * dim * 2;
    const int32_t* table = p.table + (int64_t)i * p.table_stride;
    const uint8_t* kbase = p.kc + (int64_t)kvh * dim * 2;
    const uint8_t* vbase = p.vc + (int64_t)kvh * dim * 2;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int pre = min(sp.pre, sp.seq);

    // the wave's 32 rows, one per lane column
    const int r = row0 + w * 32 + c32;
    const bool in = r < rows;
    const int tok = in ? r / G : 0, head = kvh * G + (in ? r - tok * G : 0);
    const int pos = sp.seq - sp.n + (in ? tok : (rows - 1) / G);
    const bool flip = !FEAT && p.scale < 0.f;    // a negative scale turns the queries' signs: exact
    u32x4 q[QS];
    {
        const uint8_t* src = p.q + (int64_t)(sp.first + tok) * p.q_stride + (int64_t)head * dim * 2 + h32 * 16;
#pragma unroll
        for (int s = 0; s < QS; ++s) {
            q[s] = u32x4{0, 0, 0, 0};
            if (in && (EXACT || s * 16 + h32 * 8 < dim)) q[s] = *reinterpret_cast<const u32x4*>(src + s * 32);
            if (flip) q[s] ^= 0x80008000u;
        }
    }
    // scores in units of log2: x = c s (FEAT: x computed in full, c = 1)
    const Factors by(p);
    const float c = FEAT ? 1.f : fabsf(by.log2);
    const float slope = FEAT && p.slopes != nullptr && in ? p.slopes[head] * kLog2e : 0.f;

    // the keys that the tile's rows can see
    const int p_first = sp.seq - sp.n + row0 / G, p_last = sp.seq - sp.n + min(rows - 1, row0 + kRowTile - 1) / G;
    const int key_end = max(0, min(sp.end, max(p_last + 1, pre)));
    const int key_begin = p.window > 0 ? min(key_end, max(0, p_first + 1 - p.window) / KT * KT) : 0;
    const int ntiles = key_end > key_begin ? (key_end - key_begin + KT - 1) / KT : 0;
    const int p_wave_last = __builtin_amdgcn_readfirstlane(sp.seq - sp.n + min(rows - 1, row0 + w * 32 + 31) / G);
    const int sees_to = min(max(pos + 1, pre), key_end);         // the lane's row: keys below, window aside
    const int all_see_to = __builtin_amdgcn_readfirstlane(       // every row of the wave
        min(max(sp.seq - sp.n + min(rows - 1, row0 + w * 32) / G + 1, pre), key_end));

    // The wave loads a quarter of each tile: KT / 4 rows, RPL of them per load.
    // Where pages hold whole quarters, a quarter's page id is a scalar, walked along
    // without divisions and looked up a tile ahead, and the lanes' offsets are
    // constants.  Other pages, and the tile in which the last key lies, are looked
    // up lane by lane.
    constexpr int RPL = 1024 / (DP * 2), QROWS = KT / 4;
    auto block_of = [&](int j) { return p.block_shift >= 0 ? j >> p.block_shift : j / p.block_size; };
    const __attribute__((address_space(4))) int32_t* entries = (const __attribute__((address_space(4))) int32_t*)table;
    const bool paged = p.block_size % QROWS == 0 && p.table_width > 0;
    uint32_t piece_off[Shape::LOADS];            // where in a row the lane's piece of load u starts
#pragma unroll
    for (int u = 0; u < Shape::LOADS; ++u) {
        const int piece = (lane % CPR) ^ Shape::turn(w * QROWS + lane / CPR + RPL * u);
        piece_off[u] = EXACT || piece * 8 < dim ? piece * 16 : 0;
    }
    uint32_t lane_off[Shape::LOADS];             // and in a quarter
#pragma unroll
    for (int u = 0; u < Shape::LOADS; ++u) lane_off[u] = (lane / CPR + RPL * u) * (uint32_t)row_bytes + piece_off[u];
    const int wu = __builtin_amdgcn_readfirstlane(w);
    // the quarter that is loaded next: its block, first token there, page
    int at_blk = block_of(key_begin + wu * QROWS), at_in = key_begin + wu * QROWS - at_blk * p.block_size, at_id = -1;
    const int step_blk = block_of(KT), step_in = KT - step_blk * p.block_size;
    auto look_up = [&]() { at_id = paged ? entries[min(at_blk, p.table_width - 1)] : -1; };
    auto load_tile = [&](int j0, int buf) {
        const uint32_t dst = lds0 + buf * 2 * TILE + wu * Shape::LOADS * 1024;
        if (paged && j0 + KT <= key_end) {
            const bool named = at_blk < p.table_width && (uint32_t)at_id < (uint64_t)p.num_blocks;
            if (!named) *gap = 1;
            const int64_t from = named ? ((int64_t)at_id * p.block_size + at_in) * row_bytes : 0;
#pragma unroll
            for (int u = 0; u < Shape::LOADS; ++u) {
                load_to_lds(dst + u * 1024, kbase + from, lane_off[u]);
                load_to_lds(dst + u * 1024 + TILE, vbase + from, lane_off[u]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < Shape::LOADS; ++u) {
                const int j = min(j0 + wu * QROWS + lane / CPR + RPL * u, key_end - 1), blk = block_of(j);
                const int id = blk < p.table_width ? table[blk] : -1;
                const bool named = (uint32_t)id < (uint64_t)p.num_blocks;
                if (!named) *gap = 1;
                const int64_t from = named ? ((int64_t)id * p.block_size + (j - blk * p.block_size)) * row_bytes + piece_off[u] : 0;
                load_to_lds(dst + u * 1024, kbase + from);
                load_to_lds(dst + u * 1024 + TILE, vbase + from);
            }
        }
        at_in += step_in;
        at_blk += step_blk + (at_in >= p.block_size ? 1 : 0);
        at_in -= at_in >= p.block_size ? p.block_size : 0;
        look_up();
    };
    // Where the lane's operands lie in a tile: K row c32 (+ 32 b), step k (+ 8); V^T
    // rows of its half and quarter (+ 16 k), columns d (+ 4).  Everything else
    // about an address is a constant of the unrolled loop.
    typedef const __attribute__((address_space(3))) uint8_t* lds_ptr;
    constexpr int KA = QS < 8 ? QS : 8, VA = DB < 4 ? DB : 4;
    lds_ptr ka[KA], va[2][VA];
#pragma unroll
    for (int k = 0; k < KA; ++k) ka[k] = (lds_ptr)lds + c32 * (DP * 2) + ((2 * k + h32) ^ Shape::turn(c32)) * 16;
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int d = 0; d < VA; ++d) {
            const int row = 8 * y + 4 * h32 + ((lane & 15) >> 2), piece = 4 * d + ((lane >> 4 & 1) << 1) + ((lane & 3) >> 1);
            va[y][d] = (lds_ptr)lds + row * (DP * 2) + (piece ^ Shape::turn(row)) * 16 + (lane & 1) * 8;
        }

    f32x16 acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[d][e] = 0.f;
    bool poisoned = false;
    float m = -INFINITY, l = 0.f;                // m: the scale in use, in the scores' units before c

    if (threadIdx.x == 0) *gap = 0;
    __syncthreads();
    look_up();
    if (ntiles > 0) load_tile(key_begin, 0);
    auto step = [&](auto which, int t) __attribute__((always_inline)) {
        constexpr int BUF = decltype(which)::value, K0 = BUF * 2 * TILE, V0 = K0 + TILE;
        const int j0 = key_begin + t * KT;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        const bool gaps = *gap != 0;
        if (t + 1 < ntiles) load_tile(j0 + KT, BUF ^ 1);
        if (j0 >= max(p_wave_last + 1, pre) || poisoned) return;      // nothing of the tile is seen by the wave's rows
        f32x16 s[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][e] = 0.f;
#pragma unroll
            for (int k = 0; k < QS; ++k) {
                u32x4 kf = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(ka[k & 7] + K0 + b * 32 * DP * 2 + (k >> 3) * 256);
                if (!EXACT) kf &= (2 * k + h32) * 8 < dim ? ~0u : 0u;
                s[b] = mfma32<BF16>(kf, q[k], s[b]);
            }
        }
        if constexpr (FEAT) {
            if (p.cap > 0.f) {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[b][e] = by.cap * tanh_of(s[b][e] * by.arg);
            } else {
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[b][e] *= by.log2;
            }
            if (p.slopes != nullptr) {
                const float d = (float)(pos - (j0 + 4 * h32));       // exact below 2^24, as all its steps
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        s[b][e] -= slope * fabsf(d - (float)(b * 32 + 8 * (e >> 2) + (e & 3)));
            }
        }
        const bool clear = !gaps && j0 + KT <= all_see_to && (p.window == 0 || j0 > p_wave_last - p.window);
        if (!clear) {
            uint64_t pages = ~0ull;
            if (gaps) {
                const int blk = block_of(j0 + lane);
                const int id = j0 + lane < key_end && blk < p.table_width ? table[blk] : -1;
                pages = __ballot((uint32_t)id < (uint64_t)p.num_blocks);
            }
            const int hi = sees_to - j0, lo = p.window > 0 ? pos - p.window + 1 - j0 : 0;
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                const uint32_t sees = ((uint32_t)(pages >> (32 * b)) & below(hi - 32 * b) & ~below(lo - 32 * b)) >> (4 * h32);
#pragma unroll
                for (int e = 0; e < 16; ++e) s[b][e] = (sees >> (8 * (e >> 2) + (e & 3)) & 1) ? s[b][e] : -INFINITY;
            }
            // A masked tile with infinities or NaN in V: 0 times them would reach
            // rows that do not see their key.  The wave's rows are done another way.
            uint32_t found = 0;
#pragma unroll 4
            for (int o = lane * 16; o < TILE; o += 1024)
                found |= odd_bits<BF16>(*reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((lds_ptr)lds + V0 + o));
            poisoned = __ballot(found != 0) != 0;
            if (poisoned) return;
        }
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
        top = max_across32(top);
        if (__ballot(top * c > m * c + 8.f || m == -INFINITY) != 0) {
            const float m_new = fmaxf(m, top), base = m_new == -INFINITY ? 0.f : m_new;
            const float keep = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - base) * c);
            m = m_new;
            l *= keep;
#pragma unroll
            for (int d = 0; d < DB; ++d) acc[d] *= keep;
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        u32x4 pr[2 * KB];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                f32x8 pe;
#pragma unroll
                for (int e = 0; e < 8; ++e) pe[e] = __builtin_amdgcn_exp2f(fmaf(s[b][8 * half + e], c, -mc));
                pr[2 * b + half] = round8<BF16>(pe);
                l = add_pairs<BF16>(pr[2 * b + half], l);
            }
        // V^T: among each 16 lanes, four keys by 16 columns per read
        auto v_frag = [&](int k, int d) -> u32x4 {
            const uint2 x = read_transposed(va[0][d & 3] + V0 + 16 * k * DP * 2 + (d >> 2) * 256);
            const uint2 y = read_transposed(va[1][d & 3] + V0 + 16 * k * DP * 2 + (d >> 2) * 256);
            return u32x4{x.x, x.y, y.x, y.y};
        };
        u32x4 vf[2][DB];                         // one step of 16 keys ahead
#pragma unroll
        for (int d = 0; d < DB; ++d) vf[0][d] = v_frag(0, d);
#pragma unroll
        for (int k = 0; k < 2 * KB; ++k) {
            if (k + 1 < 2 * KB) {
#pragma unroll
                for (int d = 0; d < DB; ++d) vf[(k + 1) & 1][d] = v_frag(k + 1, d);
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) acc[d] = mfma32<BF16>(vf[k & 1][d], pr[k], acc[d]);
        }
    };
    for (int t = 0; t < ntiles; t += 2) {
        step(std::integral_constant<int, 0>{}, t);
        if (t + 1 < ntiles) step(std::integral_constant<int, 1>{}, t + 1);
    }
    l = sum_across32(l);
    if (threadIdx.x == 0 && *gap != 0) raise(p.status);
    __syncthreads();                             // the tiles are done with; LDS takes the output rows
    if (poisoned) {
        for (int k = 0; k < 32 && row0 + w * 32 + k < rows; ++k) {
            const int rr = row0 + w * 32 + k, tk = rr / G, at = sp.seq - sp.n + tk;
            exact_row(p, table, sp.first + tk, kvh * G + rr - tk * G, kvh, at, p.window > 0 ? max(0, at + 1 - p.window) : 0,
                      min(sp.end, max(at + 1, pre)), lds + w * 32 * DP * 2);
        }
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint8_t* mine = lds + w * 32 * DP * 2;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            uint32_t two[2];
#pragma unroll
            for (int z = 0; z < 2; ++z)
                two[z] = (uint32_t)to_bits16(l == 0.f ? 0.f : acc[d][4 * y + 2 * z] * inv, BF16) |
                         (uint32_t)to_bits16(l == 0.f ? 0.f : acc[d][4 * y + 2 * z + 1] * inv, BF16) << 16;
            *reinterpret_cast<uint2*>(mine + c32 * (DP * 2) + ((4 * d + y) ^ (c32 & 7)) * 16 + h32 * 8) = make_uint2(two[0], two[1]);
        }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < DP / 16; ++u) {
        const int row = u * (64 / CPR) + lane / CPR, piece = lane % CPR, rr = row0 + w * 32 + row;
        if (rr < rows && (EXACT || piece * 8 < dim)) {
            const int tk = rr / G;
            const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * (DP * 2) + (piece ^ (row & 7)) * 16);
            *reinterpret_cast<u32x4*>(p.out + (int64_t)(sp.first + tk) * p.out_stride +
                                      ((int64_t)(kvh * G + rr - tk * G) * dim + piece * 8) * 2) = v;
        }
    }
}

template <int DP, bool BF16, bool EXACT, bool FEAT>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void attention_chunk_kernel(AttnParams p, Cut cut) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[ChunkShape<DP>::LDS];
    chunk_group<DP, BF16, EXACT, FEAT>(p, cut, blockIdx.x, lds);
}

// Steps of both kinds in one launch: workgroups that wait for memory and
// workgroups that wait for the matrix units share each CU.  Blocks of eight
// neighbours (one per XCD) are all of one kind, the kinds spread evenly.
template <int DP, bool BF16, bool EXACT, bool FEAT>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void attention_mixed_kernel(AttnParams p, Partial part, Cut cut) {
    constexpr int LDS = ChunkShape<DP>::LDS > kRowsLds<DP, 1> ? ChunkShape<DP>::LDS : kRowsLds<DP, 1>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
    const int64_t b = blockIdx.x >> 3, tiles = (cut.tile_groups + 7) >> 3, all = tiles + ((cut.row_groups + 7) >> 3);
    const int before = (int)(b * tiles / all), after = (int)((b + 1) * tiles / all);
    if (after > before) {
        const int group = before * 8 + (blockIdx.x & 7);
        if (group < cut.tile_groups) chunk_group<DP, BF16, EXACT, FEAT>(p, cut, group, lds);
    } else {
        const int group = ((int)b - before) * 8 + (blockIdx.x & 7);
        if (group < cut.row_groups) rows_group<DP, 1, BF16, EXACT>(p, part, cut, group, lds);
    }
}

namespace {

// How a call is cut: by what the host knows, and for every length that the
// device may hold.
struct Plan {
    Cut cut;
    int nb;              // 16-row blocks of the few-rows part, 0: no such part
    bool chunks;         // some request may be larger
    bool together;       // both parts in one launch
    int dp;              // head size of the kernels
    int most_splits;     // bound of cut.splits for any window and prefix (workspaces go by it)
};

constexpr int kTargetGroups = 1024;      // workgroups that keep 256 CUs evenly busy
constexpr int kMinSplitLen = 256;

Plan plan_of(const AttnParams& p) {
    Plan r{};
    const int G = p.heads / p.kv_heads;
    const int64_t most = (int64_t)std::max(p.max_q, 1) * G;
    r.dp = p.dim <= 64 ? 64 : p.dim <= 128 ? 128 : 256;
    // Requests of up to 64 rows per K/V head take the few-rows kernel; beside
    // larger ones, those of a single token do.
    const int64_t few = most <= 64 ? most : G <= 64 ? G : 0;
    r.chunks = most > 64;
    r.nb = few == 0 ? 0 : few <= 16 ? 1 : few <= 32 ? 2 : 4;
    Cut& c = r.cut;
    c.row_limit = 16 * r.nb;
    c.max_rows = (int)std::min<int64_t>(most, c.row_limit);
    const int64_t keys = p.window > 0 && p.prefix == nullptr ? std::min<int64_t>(p.max_seq, (int64_t)p.window + p.max_q + 31) : p.max_seq;
    const int64_t groups = std::max<int64_t>(1, (int64_t)p.num_reqs * p.kv_heads);
    const int64_t want = std::max<int64_t>(1, kTargetGroups / groups);
    // One launch for both parts where there may be enough single tokens to fill the
    // card (124 requests of 8 K/V heads, 4 of them chunks: 755 us against 774 in two
    // launches); two where there are few requests (4 chunks: 2070 us against 2260).
    // A grid of both kinds has to stay below 2^32 lanes as well.
    const int64_t tiles = ((int64_t)p.num_tokens * G / kRowTile + p.num_reqs) * p.kv_heads;
    r.together = r.chunks && r.nb == 1 && groups >= 512 && tiles + 16 * groups < (1 << 24) - 16;
    // Pieces of no more than 8192 keys, so that one long request does not outlast the
    // others; beside chunks 2048, as the two kinds' groups end together (mixed step
    // 755 us; pieces of 4096 831, of 1024 800).  256 requests of up to 4096 keys take
    // 434 us uncut, 528 in pieces of 2048 and 562 in pieces of 1024.
    const int64_t longest = r.together ? 2048 : 8192;
    c.min_len = (int)std::min<int64_t>(longest, std::max<int64_t>(kMinSplitLen, ((keys + want - 1) / want + 31) / 32 * 32));
    c.splits = (int)std::max<int64_t>(1, std::min<int64_t>((keys + c.min_len - 1) / c.min_len, std::min<int64_t>(std::max<int64_t>(want, 16), 256)));
    // fewer keys (a window) are cut into at most `want` pieces of at least kMinSplitLen
    const int64_t all = std::max<int64_t>(p.max_seq, 1);
    r.most_splits = (int)std::max<int64_t>({c.splits, std::min(want, (all + kMinSplitLen - 1) / kMinSplitLen),
                                            std::min<int64_t>((all + longest - 1) / longest, std::max<int64_t>(want, 16))});
    r.most_splits = std::min(r.most_splits, 256);
    c.row_groups = r.nb > 0 ? p.num_reqs * c.splits * p.kv_heads : 0;
    c.tile_groups = r.chunks ? (int)tiles : 0;
    return r;
}

int64_t partial_rows(const AttnParams& p, const Plan& r) {
    return r.nb > 0 && r.cut.splits > 1 ? (int64_t)p.num_reqs * p.kv_heads * r.cut.max_rows * r.cut.splits : 0;
}

template <int DP, bool BF16, bool EXACT>
void launch(const AttnParams& p, const Plan& r, Partial part, hipStream_t s) {
    const Cut& c = r.cut;
    // caps, biases and a scale of zero need the whole score before the mask
    const bool feat = p.cap > 0.f || p.slopes != nullptr || p.scale == 0.f;
    if (r.together) {
        const dim3 grid(((c.tile_groups + 7) / 8 + (c.row_groups + 7) / 8) * 8);
        if (feat) hipLaunchKernelGGL((attention_mixed_kernel<DP, BF16, EXACT, true>), grid, dim3(256), 0, s, p, part, c);
        else hipLaunchKernelGGL((attention_mixed_kernel<DP, BF16, EXACT, false>), grid, dim3(256), 0, s, p, part, c);
    } else {
        if (r.nb == 1) hipLaunchKernelGGL((attention_rows_kernel<DP, 1, BF16, EXACT>), dim3(c.row_groups), dim3(256), 0, s, p, part, c);
        if (r.nb == 2) hipLaunchKernelGGL((attention_rows_kernel<DP, 2, BF16, EXACT>), dim3(c.row_groups), dim3(256), 0, s, p, part, c);
        if (r.nb == 4) hipLaunchKernelGGL((attention_rows_kernel<DP, 4, BF16, EXACT>), dim3(c.row_groups), dim3(256), 0, s, p, part, c);
        if (r.chunks && feat) hipLaunchKernelGGL((attention_chunk_kernel<DP, BF16, EXACT, true>), dim3(c.tile_groups), dim3(256), 0, s, p, c);
        if (r.chunks && !feat) hipLaunchKernelGGL((attention_chunk_kernel<DP, BF16, EXACT, false>), dim3(c.tile_groups), dim3(256), 0, s, p, c);
    }
    if (r.nb > 0 && c.splits > 1)
        hipLaunchKernelGGL((join_rows_kernel<DP>), dim3(p.num_reqs, p.kv_heads * c.max_rows), dim3(256), 0, s, p, part, c);
}

}  // namespace

size_t attention_workspace(const AttnParams& p) {
    const Plan r = plan_of(p);
    if (r.nb == 0 || r.most_splits <= 1) return 0;
    return (size_t)p.num_reqs * p.kv_heads * r.cut.max_rows * r.most_splits * (r.dp * 4 + 8);
}

hipError_t launch_attention(const AttnParams& p, void* workspace, hipStream_t s) {
    const Plan r = plan_of(p);
    Partial part{};
    part.o = static_cast<float*>(workspace);
    part.ml = reinterpret_cast<float2*>(part.o + partial_rows(p, r) * r.dp);
    auto with = [&](auto dp, auto bf16) {
        if (p.dim == decltype(dp)::value) launch<decltype(dp)::value, decltype(bf16)::value, true>(p, r, part, s);
        else launch<decltype(dp)::value, decltype(bf16)::value, false>(p, r, part, s);
    };
    auto by_dim = [&](auto bf16) {
        if (r.dp == 64) with(std::integral_constant<int, 64>{}, bf16);
        else if (r.dp == 128) with(std::integral_constant<int, 128>{}, bf16);
        else with(std::integral_constant<int, 256>{}, bf16);
    };
    if (p.bf16) by_dim(std::true_type{}); else by_dim(std::false_type{});
    return hipGetLastError();
}

}  // namespace ric
