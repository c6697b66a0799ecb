// Log probabilities of given tokens, their rank, the row's entropy and the top
// alternatives.  With a reference m (the row's maximum, or a value up to 2^8 times
// less likely), S = sum e^(x-m) and W = sum e^(x-m) (x-m):
//     logprob = x_t - m - ln S,   entropy = ln S - W / S
// Sums are float32, per lane, then across lanes, waves and pieces in a fixed order.
//
// Tokens are ordered by (logit descending, id ascending), which a 64-bit key
// holds: the logit's bits mapped to an increasing unsigned number above the
// complement of the id.  -0 counts as +0, a NaN lies above everything.
//
// Bound by reading the logits once: one pass, 16 bytes per lane and load, the next
// block's loads in flight while a block is summed.  Rows are cut into pieces,
// one workgroup each, where there are few of them.
#include <algorithm>

#include "ric_internal.h"

namespace ric {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kVectors = 2;                  // loads of 16 bytes per lane and block

struct Piece {                               // one piece of a row
    float m, S, W;                           // sums relative to m, W in units of log2
    int above;                               // tokens ordered before the target
};

template <int DT>
__device__ __forceinline__ float load_logit(const uint8_t* row, int64_t i) {
    if constexpr (DT == 2) return reinterpret_cast<const float*>(row)[i];
    const uint16_t h = reinterpret_cast<const uint16_t*>(row)[i];
    if constexpr (DT == 1) return __uint_as_float((uint32_t)h << 16);
    return (float)__builtin_bit_cast(_Float16, h);
}

// Element e of a 16-byte vector.
template <int DT>
__device__ __forceinline__ float element(u32x4 v, int e) {
    if constexpr (DT == 2) return __uint_as_float(v[e]);
    const uint32_t two = v[e >> 1];
    if constexpr (DT == 1) return __uint_as_float((e & 1) ? two & 0xffff0000u : two << 16);
    const uint16_t h = (uint16_t)((e & 1) ? two >> 16 : two);
    return (float)__builtin_bit_cast(_Float16, h);
}

__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
// The next float below x (> -inf).
__device__ __forceinline__ float lower_than(float x) {
    const uint32_t o = ordered(x);
    return from_ordered(o == 0x80000000u ? 0x7ffffffeu : o - 1);     // -0 is 0
}
// The next float above x (< inf).
__device__ __forceinline__ float higher_than(float x) {
    const uint32_t o = ordered(x);
    return from_ordered(o == 0x7ffffffeu ? 0x80000000u : o + 1);
}
__device__ __forceinline__ u64 key_of(float x, int id) { return (u64)ordered(x) << 32 | (uint32_t)~id; }
__device__ __forceinline__ int id_of(u64 key) { return (int)~(uint32_t)key; }

__device__ __forceinline__ u64 read_lane(u64 x, int lane) {
    return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
}

// The value of lane ^ O, in vector moves (an exchange through LDS takes several
// times as long, and the sorts below are chains of them).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return __builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int O>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
    constexpr int kQuad1032 = 0xb1, kQuad2301 = 0x4e, kQuad3210 = 0x1b, kMirror = 0x140, kHalfMirror = 0x141;
    const int lane = threadIdx.x & 63;
    if constexpr (O == 1) return dpp<kQuad1032>(x);
    else if constexpr (O == 2) return dpp<kQuad2301>(x);
    else if constexpr (O == 4) return dpp<kQuad3210>(dpp<kHalfMirror>(x));
    else if constexpr (O == 8) return dpp<kHalfMirror>(dpp<kMirror>(x));
    else if constexpr (O == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        return (lane & 16) ? r[0] : r[1];
    } else if constexpr (O == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return (lane & 32) ? r[0] : r[1];
    } else {
        static_assert(O == 63);
        return lane_xor<32>(lane_xor<16>(dpp<kMirror>(x)));
    }
}
template <int O>
__device__ __forceinline__ float lane_xor(float x) { return __uint_as_float(lane_xor<O>(__float_as_uint(x))); }
template <int O>
__device__ __forceinline__ u64 lane_xor(u64 x) {
    return (u64)lane_xor<O>((uint32_t)(x >> 32)) << 32 | lane_xor<O>((uint32_t)x);
}

// One step of a bitonic sort: lanes O apart, descending where DESC.
template <int O, class T>
__device__ __forceinline__ T exchange(T x, bool larger) {
    const T y = lane_xor<O>(x);
    return larger == (y > x) ? y : x;
}
template <int K, int O, class T>
__device__ __forceinline__ T sort_steps(T x) {
    const int lane = threadIdx.x & 63;
    x = exchange<O>(x, ((lane & O) == 0) == ((lane & K) == 0));
    if constexpr (O > 1) return sort_steps<K, O / 2>(x);
    else return x;
}
// The lanes' values in descending order.
template <class T>
__device__ __forceinline__ T sort64(T x) {
    x = sort_steps<2, 1>(x);
    x = sort_steps<4, 2>(x);
    x = sort_steps<8, 4>(x);
    x = sort_steps<16, 8>(x);
    x = sort_steps<32, 16>(x);
    return sort_steps<64, 32>(x);
}

// A wave's best keys so far, in descending order over its lanes (0: none).
__device__ __forceinline__ void insert(u64& best, u64 key) {
    const int at = __popcll(__ballot(best > key));
    constexpr int kWaveShr1 = 0x138;
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)best, kWaveShr1, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(best >> 32), kWaveShr1, 0xf, 0xf, false);
    const int lane = threadIdx.x & 63;
    best = lane < at ? best : lane == at ? key : ((u64)hi << 32 | lo);
}

// Joins two descending lists: the larger of each lane and the other list's mirror
// holds the best 64 as a bitonic sequence, which six exchanges sort.
__device__ __forceinline__ u64 join(u64 a, u64 b) {
    return sort_steps<64, 32>(max(a, lane_xor<63>(b)));
}

__device__ __forceinline__ float wave_sum(float x) {
    x += lane_xor<1>(x);
    x += lane_xor<2>(x);
    x += lane_xor<4>(x);
    x += lane_xor<8>(x);
    x += lane_xor<16>(x);
    return x + lane_xor<32>(x);
}

// Adds piece b to piece a.
__device__ __forceinline__ void add(Piece& a, const Piece& b) {
    const float m = fmaxf(a.m, b.m), base = m == -INFINITY ? 0.f : m;
    // e^(x-m) (x-m) moves to a new reference as f (W + d S)
    const float da = a.m == -INFINITY ? 0.f : (a.m - base) * kLog2e, db = b.m == -INFINITY ? 0.f : (b.m - base) * kLog2e;
    const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
    // a reference so far below that its weights vanish has nothing to move
    a.W = (fa == 0.f ? 0.f * a.S : fa * fmaf(da, a.S, a.W)) + (fb == 0.f ? 0.f * b.S : fb * fmaf(db, b.S, b.W));
    a.S = a.S * fa + b.S * fb;
    a.m = m;
    a.above += b.above;
}

// A row with NaN or infinities above: every log probability is NaN, the order is
// found token by token, one pass per alternative.  256 threads.
template <int DT>
__device__ void broken_row(const LogprobParams& p, int r, const uint8_t* row, u64* shared) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    auto block = [&](u64 k, bool sum) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const u64 y = __shfl_xor(k, o);
            k = sum ? k + y : max(k, y);
        }
        __syncthreads();
        if (lane == 0) shared[w] = k;
        __syncthreads();
        return sum ? shared[0] + shared[1] + shared[2] + shared[3] : max(max(shared[0], shared[1]), max(shared[2], shared[3]));
    };
    const int target = p.targets != nullptr ? p.targets[r] : -1;
    const bool has = target >= 0 && target < p.vocab;
    const u64 kt = has ? key_of(load_logit<DT>(row, target), target) : 0;
    u64 above = 0, last = ~0ull;
    for (int i = threadIdx.x; i < p.vocab; i += 256) above += has && key_of(load_logit<DT>(row, i), i) > kt;
    above = block(above, true);
    if (threadIdx.x == 0) {
        if (p.targets != nullptr) {
            p.logprob[r] = has ? NAN : 0.f;
            p.rank[r] = has ? 1 + (int)above : 0;
        }
        if (p.entropy != nullptr) p.entropy[r] = NAN;
    }
    for (int k = 0; k < p.top_k; ++k) {
        u64 b = 0;
        for (int i = threadIdx.x; i < p.vocab; i += 256) {
            const u64 c = key_of(load_logit<DT>(row, i), i);
            if (c < last) b = max(b, c);
        }
        last = block(b, false);
        if (threadIdx.x == 0) {
            p.top_ids[(int64_t)r * p.top_k + k] = id_of(last);
            p.top_logprobs[(int64_t)r * p.top_k + k] = NAN;
        }
    }
}

// Writes row r from its whole piece and best keys; called by 256 threads, the
// keys in the lanes of the first wave.
template <int DT>
__device__ __forceinline__ void finish_row(const LogprobParams& p, int r, const uint8_t* row, const Piece& whole, u64 best,
                                           u64* shared) {
    const int target = p.targets != nullptr ? p.targets[r] : -1;
    if (threadIdx.x == 0 && target >= p.vocab && p.status != nullptr) atomicAdd(p.status, 1);
    if (whole.S != whole.S) {
        broken_row<DT>(p, r, row, shared);
        return;
    }
    if (threadIdx.x >= 64) return;
    const bool none = whole.m == -INFINITY;      // no token has a probability
    const float lnS = logf(whole.S);
    if (threadIdx.x == 0) {
        const bool has = target >= 0 && target < p.vocab;
        if (p.targets != nullptr) {
            p.logprob[r] = !has ? 0.f : none ? -INFINITY : (load_logit<DT>(row, target) - whole.m) - lnS;
            p.rank[r] = has ? 1 + whole.above : 0;
        }
        if (p.entropy != nullptr) p.entropy[r] = none ? 0.f : lnS - whole.W * kLn2 / whole.S;
    }
    if ((int)threadIdx.x < p.top_k) {
        const int64_t at = (int64_t)r * p.top_k + threadIdx.x;
        p.top_ids[at] = id_of(best);
        p.top_logprobs[at] = none ? -INFINITY : (from_ordered((uint32_t)(best >> 32)) - whole.m) - lnS;
    }
}

}  // namespace

// One piece of a row per workgroup: its 16-byte vectors in blocks of 64 lanes x
// kVectors, dealt to the four waves in turn, so that a wave meets rising ids.
// A row may start at any element: those before the first whole vector go to the
// first piece's first wave before its blocks, those behind the last to the last
// piece's after them.
//   m: a wave takes its first block's maximum, and a new one where a block exceeds
//     it by more than 2^8, so hardly any block rescales.
//   top: a wave keeps its best keys sorted over its lanes; a block is looked at again
//     only if its maximum reaches the floor: the wave's own K-th key, or the least
//     of the four waves' ceil(K / 4)-th, which K tokens of the row reach together.
//     Over unsorted tokens that happens about K / 4 ln(n / K) times per wave.  What
//     passes is entered one by one, or sorted and joined where it is many.  The first
//     block is entered above the K-th largest of its lanes' maxima.
//   rank: a compare and a count of the lanes per 64 tokens; equal logits count
//     before the target's id, so blocks before it compare with the next lower float.
// 64 registers: eight workgroups share a CU and keep its loads in flight (with blocks
// of twice the size and six workgroups the same rows take 3 to 5% longer).
// Measured (bf16): 2048 rows of 152064 with 5 alternatives 147 us, 4.25 TB/s (110 us,
// 5.5 TB/s, without target and alternatives); 256 rows of 128256 with 20, 35 + 5 us.
template <int DT>
__global__ __launch_bounds__(256, 8) void logprobs_kernel(LogprobParams p, int pieces, Piece* part, u64* part_keys) {
    constexpr int VE = DT == 2 ? 4 : 8;          // elements per vector
    constexpr int BLOCK = 64 * kVectors;         // vectors per block
    __shared__ Piece waves[4];
    __shared__ u64 lists[4][64];
    __shared__ float quarters[4];                // the waves' ceil(K / 4)-th values so far
    const int r = blockIdx.x / pieces, piece = blockIdx.x - r * pieces;
    const int count = p.dev_count != nullptr ? min(p.max_rows, *p.dev_count) : p.max_rows;
    if (r >= count) return;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint8_t* row = p.logits + (int64_t)r * p.row_stride;
    const int size = DT == 2 ? 4 : 2;
    const int head = min(p.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / size);
    const int vectors = (p.vocab - head) / VE, tail = p.vocab - head - vectors * VE;
    const u32x4* body = reinterpret_cast<const u32x4*>(row + (int64_t)head * size);
    const int blocks = (vectors + BLOCK - 1) / BLOCK;
    const int b0 = (int)((int64_t)blocks * piece / pieces), b1 = (int)((int64_t)blocks * (piece + 1) / pieces);
    u32x4 now[kVectors];
    auto request = [&](int b) {
#pragma unroll
        for (int u = 0; u < kVectors; ++u)
            now[u] = body[min(b * BLOCK + u * 64 + lane, vectors - 1)];
    };
    if (b0 + w < b1) request(b0 + w);            // under way while the target is looked up
    const int target = p.targets != nullptr ? p.targets[r] : -1;
    const bool has = target >= 0 && target < p.vocab;
    const float xt = has ? load_logit<DT>(row, target) : INFINITY;
    // x >= xt is x > lower (for xt = -inf, every x)
    const float lower = xt == -INFINITY ? xt : lower_than(xt);
    const int K = p.top_k;

    Piece mine{-INFINITY, 0.f, 0.f, 0};          // S and W are the lane's own
    u64 best = 0;
    float floor_x = -INFINITY;                   // value of the K-th best key
    bool open = K > 0;                           // fewer than K keys yet
    if (threadIdx.x < 4) quarters[threadIdx.x] = -INFINITY;
    __syncthreads();
    auto enter = [&](u64 key, u64 lanes) {       // the keys of these lanes
        if (__popcll(lanes) > 12) {
            best = join(best, sort64((lanes >> lane & 1) ? key : 0));
        } else {
            for (; lanes != 0; lanes &= lanes - 1) {
                const u64 one = read_lane(key, __ffsll(lanes) - 1);
                if (one > read_lane(best, K - 1)) insert(best, one);
            }
        }
    };
    auto settle = [&]() {
        const u64 kth = read_lane(best, K - 1);
        open = kth == 0;
        floor_x = open ? -INFINITY : from_ordered((uint32_t)(kth >> 32));
        const u64 quarter = read_lane(best, (K + 3) / 4 - 1);
        if (lane == 0 && quarter != 0) *(volatile float*)&quarters[w] = from_ordered((uint32_t)(quarter >> 32));
    };
    auto weigh = [&](float x) {
        const float d = (x - (mine.m == -INFINITY ? 0.f : mine.m)) * kLog2e;
        const float e = __builtin_amdgcn_exp2f(d);
        mine.S += e;
        mine.W = fmaf(e, fmaxf(d, -300.f), mine.W);      // 0 * -inf has no place in W
    };
    auto refer = [&](float top) {                // `top`: the wave's largest new logit
        if (top <= mine.m + 8.f * kLn2 || top == -INFINITY) return;
        const float d = mine.m == -INFINITY ? 0.f : (mine.m - top) * kLog2e, f = __builtin_amdgcn_exp2f(d);
        mine.W = f == 0.f ? 0.f * mine.S : f * fmaf(d, mine.S, mine.W);
        mine.S *= f;
        mine.m = top;
    };
    auto wave_max = [&](float x) {
        x = fmaxf(x, lane_xor<1>(x));
        x = fmaxf(x, lane_xor<2>(x));
        x = fmaxf(x, lane_xor<4>(x));
        x = fmaxf(x, lane_xor<8>(x));
        x = fmaxf(x, lane_xor<16>(x));
        return fmaxf(x, lane_xor<32>(x));
    };
    auto loose = [&](int first, int n) {         // n < 8 single elements
        const bool in = lane < n;
        const int id = first + lane;
        const float x = in ? load_logit<DT>(row, id) : -INFINITY;
        refer(wave_max(x));
        if (in) weigh(x);
        mine.above += __popcll(__ballot(in && has && (x > xt || (x == xt && id < target))));
        if (K > 0) {
            enter(key_of(x, id), __ballot(in));
            settle();
        }
    };

    if (w == 0 && piece == 0 && head > 0) loose(0, head);
    for (int b = b0 + w; b < b1; b += 4) {
        const bool whole_block = (b + 1) * BLOCK <= vectors;
        if (!whole_block) {                      // the row's last: lanes past its end see nothing
#pragma unroll
            for (int u = 0; u < kVectors; ++u)
                if (b * BLOCK + u * 64 + lane >= vectors) {
                    const uint32_t low = DT == 2 ? 0xff800000u : DT == 1 ? 0xff80ff80u : 0xfc00fc00u;
                    now[u] = u32x4{low, low, low, low};
                }
        }
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kVectors; ++u)
#pragma unroll
            for (int e = 0; e < VE; ++e) top = fmaxf(top, element<DT>(now[u], e));
        if (__ballot(top > mine.m + 8.f * kLn2) != 0) refer(wave_max(top));
#pragma unroll
        for (int u = 0; u < kVectors; ++u)
#pragma unroll
            for (int e = 0; e < VE; ++e) weigh(element<DT>(now[u], e));
        const int id0 = head + b * BLOCK * VE;   // the block's first id
        if (has) {
            if (target < id0 || (target >= id0 + BLOCK * VE && xt != -INFINITY)) {
                const float past = target < id0 ? xt : lower;
#pragma unroll
                for (int u = 0; u < kVectors; ++u)
#pragma unroll
                    for (int e = 0; e < VE; ++e) mine.above += __popcll(__ballot(element<DT>(now[u], e) > past));
            } else if (target >= id0 + BLOCK * VE) {
                mine.above += BLOCK * VE;        // every token is at least -inf
            } else {
#pragma unroll 1
                for (int k = lane; k < BLOCK * VE; k += 64) {
                    const int id = id0 + k;
                    const float x = id < head + vectors * VE ? load_logit<DT>(row, id) : -INFINITY;
                    mine.above += __popcll(__ballot(id < head + vectors * VE && (x > xt || (x == xt && id < target))));
                }
            }
        }
        float shared_floor = -INFINITY;
        if (K > 0) {
            const volatile float* q = quarters;
            shared_floor = fminf(fminf(q[0], q[1]), fminf(q[2], q[3]));
        }
        if (K > 0 && (open || __ballot(top > floor_x && top >= shared_floor) != 0)) {
            // Tokens of the wave's earlier blocks have lower ids: these must exceed
            // their K-th; of other waves' tokens nothing is known.
            float reach = shared_floor;          // tokens >= reach pass
            if (open && whole_block) {
                // 64 lanes' maxima, sorted: at least K tokens reach the K-th of them
                const float x = sort64(top);
                reach = fmaxf(reach, __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), K - 1)));
            } else if (!open && floor_x >= reach) {
                reach = higher_than(floor_x);
            }
            // the lane's passing tokens, as bits; each is read again and entered
            uint32_t passing = 0;
#pragma unroll
            for (int u = 0; u < kVectors; ++u)
#pragma unroll
                for (int e = 0; e < VE; ++e) passing |= element<DT>(now[u], e) >= reach ? 1u << (u * VE + e) : 0u;
            if (!whole_block) {
#pragma unroll
                for (int u = 0; u < kVectors; ++u)
                    if (b * BLOCK + u * 64 + lane >= vectors) passing &= ~(((1u << VE) - 1u) << (u * VE));
            }
            for (u64 lanes = __ballot(passing != 0); lanes != 0; lanes = __ballot(passing != 0)) {
                const int k = __ffs(passing) - 1;
                const int id = id0 + ((k / VE) * 64 + lane) * VE + k % VE;
                enter(passing != 0 ? key_of(load_logit<DT>(row, id), id) : 0, lanes);
                passing &= passing - 1;
            }
            settle();
        }
        if (b + 4 < b1) request(b + 4);
    }
    if (w == 0 && piece == pieces - 1 && tail > 0) loose(head + vectors * VE, tail);

    mine.S = wave_sum(mine.S);
    mine.W = wave_sum(mine.W);
    if (lane == 0) waves[w] = mine;
    lists[w][lane] = best;
    __syncthreads();
    Piece whole = waves[0];
    for (int k = 1; k < 4; ++k) add(whole, waves[k]);
    if (w == 0 && K > 0) {
#pragma unroll 1
        for (int k = 1; k < 4; ++k) best = join(best, lists[k][lane]);
    }
    if (pieces == 1) {
        __syncthreads();
        finish_row<DT>(p, r, row, whole, best, &lists[0][0]);
        return;
    }
    if (w != 0) return;
    const int64_t at = (int64_t)r * pieces + piece;
    if (lane == 0) part[at] = whole;
    if (lane < K) part_keys[at * K + lane] = best;
}

// Joins the pieces of a row (at most 32): sums in a tree over the lanes, key lists
// one after the other, the next one's load in flight.
template <int DT>
__global__ __launch_bounds__(256) void logprobs_join_kernel(LogprobParams p, int pieces, const Piece* part, const u64* part_keys) {
    __shared__ u64 shared[4];
    const int r = blockIdx.x, lane = threadIdx.x & 63;
    const int count = p.dev_count != nullptr ? min(p.max_rows, *p.dev_count) : p.max_rows;
    if (r >= count) return;
    const u64* keys = part_keys + (int64_t)r * pieces * p.top_k;
    const bool mine = threadIdx.x < 64 && lane < p.top_k;
    u64 best = 0, next = mine ? keys[lane] : 0;
    Piece whole{-INFINITY, 0.f, 0.f, 0};
    if (lane < pieces) whole = part[(int64_t)r * pieces + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Piece other{__shfl_xor(whole.m, o), __shfl_xor(whole.S, o), __shfl_xor(whole.W, o), __shfl_xor(whole.above, o)};
        if (lane & o) {                          // the same operands in the same order on both sides
            Piece sum = other;
            add(sum, whole);
            whole = sum;
        } else {
            add(whole, other);
        }
    }
    whole = Piece{__shfl(whole.m, 0), __shfl(whole.S, 0), __shfl(whole.W, 0), __shfl(whole.above, 0)};
    if (threadIdx.x < 64 && p.top_k > 0)
        for (int k = 0; k < pieces; ++k) {
            const u64 now = next;
            next = mine && k + 1 < pieces ? keys[(int64_t)(k + 1) * p.top_k + lane] : 0;
            best = k == 0 ? now : join(best, now);
        }
    finish_row<DT>(p, r, p.logits + (int64_t)r * p.row_stride, whole, best, shared);
}

namespace {

// Pieces per row: enough workgroups to fill 256 CUs four times over, each with at
// least 8192 logits.
int pieces_of(int32_t max_rows, int32_t vocab) {
    const int want = (1024 + max_rows - 1) / max_rows;
    return std::max(1, std::min({want, vocab / 8192, 32}));
}

template <int DT>
hipError_t launch(const LogprobParams& p, Piece* part, u64* keys, int pieces, hipStream_t s) {
    hipLaunchKernelGGL(logprobs_kernel<DT>, dim3(p.max_rows * pieces), dim3(256), 0, s, p, pieces, part, keys);
    if (pieces > 1) hipLaunchKernelGGL(logprobs_join_kernel<DT>, dim3(p.max_rows), dim3(256), 0, s, p, pieces, part, keys);
    return hipGetLastError();
}

}  // namespace

size_t logprobs_workspace(int32_t max_rows, int32_t vocab, int32_t top_k) {
    return pieces_of(max_rows, vocab) == 1 ? 0 : (size_t)max_rows * pieces_of(max_rows, vocab) * (sizeof(Piece) + 8 * (size_t)top_k);
}

size_t logprobs_workspace_up_to(int32_t max_rows, int32_t vocab, int32_t top_k) {
    // r <= max_rows rows in min(ceil(1024 / r), most) pieces each, none where that is 1
    const int64_t rows = std::min(max_rows, 1023), most = std::min(vocab / 8192, 32);
    return most <= 1 ? 0 : (size_t)std::min(rows * most, rows + 1023) * (sizeof(Piece) + 8 * (size_t)top_k);
}

hipError_t launch_logprobs(const LogprobParams& p, void* workspace, hipStream_t s) {
    const int pieces = pieces_of(p.max_rows, p.vocab);
    Piece* part = static_cast<Piece*>(workspace);
    u64* keys = reinterpret_cast<u64*>(part + (int64_t)p.max_rows * pieces);
    if (p.dtype == 2) return launch<2>(p, part, keys, pieces, s);
    if (p.dtype == 1) return launch<1>(p, part, keys, pieces, s);
    return launch<0>(p, part, keys, pieces, s);
}

}  // namespace ric
