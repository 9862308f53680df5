// moe_topk.cu - the experts of each token and their gating weights from the
// logits of any number of tokens (moe_topk), and the weights' gradient back to
// the logits (moe_topk_grad).
//
// A warp takes a row, VEC * J values a lane.  A logit becomes a 32-bit key whose
// unsigned order is the choice's: larger numbers first, -0 equal to 0, NaN above
// all.  The choice works on keys whose 10 lowest bits are replaced by the expert's
// index (reversed, so that the lower one wins): one maximum over the warp then names
// the value and who holds it, no two keys are equal, and a lane keeps its four
// largest in order, so that a round is a maximum and a step of the lane that had
// it.  A row where this may not be exact is done again with whole keys
// (choose_exactly): two of the k + 1 largest that agree in their upper 22 bits (fp32
// logits: about two rows in a hundred; bf16 ones are exact), or four of the chosen in
// one lane (8 of 256: four rows in a thousand; 32 of 1024: half of them).
// 65536 rows of 256 in fp32, 8 chosen, take 26.2 us on the device so (298 instructions
// a row, the integer pipe 63% busy), 63.6 when every round looked through all values
// of its lane.  Many rows of up to 512, of which up to eight are chosen, go four to a
// warp (topk_quad_kernel): x 512 28.3 us (38.9 with a warp a row), x 256 19.9 (26.2),
// x 128 15.2 (19.3), x 64 12.2 (18.7); in bf16 19.6 (34.6), 14.1 (23.7), 13.7 (16.8),
// 11.2 (16.8).  No unit is full there (x 256 in fp32: 54% of the issue slots, the integer
// pipe at 69%, DRAM at 39%): warps wait, most for the chosen pieces and then the chosen
// logits, which are read again one behind the other.  The gradient moves more and decides
// less: 65536 x 128 in bf16 over all E 12.1 us (4.5 TB/s), 60% of the issue slots; it
// waits for shared memory, which it uses value by value.
#include <cuda_bf16.h>
#include <math.h>

#include "moe_around.h"
#include "moe_launch.h"
#include "moe_router.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xFFFFFFFFu;
// blocks of a launch that share an SM (registers for the rows in hand); of the gradient, with one row more
constexpr int grad_blocks(int values, bool row) {
    return values <= 4 ? 5 : values <= 8 ? 4 : values <= 16 ? (row ? 2 : 3) : 1;
}
constexpr int blocks_per_sm(int values) { return values <= 4 ? 6 : values <= 8 ? 5 : values <= 16 ? 3 : 2; }

constexpr int quad_blocks(int pieces, int bytes) {
    return pieces <= 2 ? 5 : pieces <= 4 || (pieces <= 8 && bytes == 2) ? 4 : pieces <= 8 ? 3 : 2;
}

constexpr uint32_t kNone = 0x007FFFFFu;   // the key of -inf: what is not above it may not be taken
constexpr uint32_t kIndex = MOE_MAX_EXPERTS - 1;

__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);   // -0 becomes 0, a NaN the positive one
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float sigmoid(float l) {
    const float z = expf(-fabsf(l));
    return __fdividef(l < 0.f ? z : 1.f, 1.f + z);   // (a NaN stays one)
}
// sigma(l) exp(-m) for the row's largest m < 0: what all of a row's sigmas have in common cancels in their ratios, so that
// rows whose sigmas would vanish keep theirs
__device__ __forceinline__ float sigmoid_over(float l, float m) { return expf(l - m) / (1.f + expf(l)); }

// sums and maxima over L lanes side by side (a NaN is the largest)
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    if constexpr (L == 32) {
        return warp_max(v);
    } else {
#pragma unroll
        for (int off = L / 2; off >= 1; off >>= 1) v = max_nan(v, __shfl_xor_sync(kAll, v, off));
        return v;
    }
}

// a row of logits in L lanes; past E, where load does not come, it is -inf
template <typename T, int VEC, int J, int L = 32>
struct Row {
    Raw<T, VEC> v[J];
    __device__ __forceinline__ Row() {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < (int)(sizeof(v[j].w) / 4); ++i) v[j].w[i] = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
    }
    __device__ __forceinline__ void load(const T *row, int E, int lane) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = L * VEC * j + VEC * lane;
            if (e < E) v[j].load(row + e);
        }
    }
    __device__ __forceinline__ float value(int i) const { return v[i / VEC].value(i % VEC); }   // i: of VEC * J
    // sum of exp(l - m)
    __device__ __forceinline__ float sum(float m) const {
        constexpr int RUN = VEC * J < 32 ? VEC * J : 32;   // (no more additions in turn)
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VEC * J; i += RUN) {
            float part = 0.f;
#pragma unroll
            for (int k = 0; k < RUN; ++k) part += exp_fast(value(i + k) - m);
            s = i ? s + part : part;
        }
        return lanes_sum<L>(s);
    }
};

// of four; a NaN is the largest
__device__ __forceinline__ float largest(const Raw<float, 4> &r) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(r.value(0)), "f"(r.value(1)), "f"(r.value(2)));
    return max_nan(m, r.value(3));
}
__device__ __forceinline__ float largest(const Raw<__nv_bfloat16, 4> &r) {
    uint32_t m;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(r.w[0]), "r"(r.w[1]));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}

// A row's slots lie in `width` lanes side by side, each with a chosen logit (-inf: none); m: the row's largest, all: sum of
// exp(l - m) over the row where the weights are shares of it.  The slot's weight; slope: 1 - sigma(l), or 1 for softmax.
__device__ __forceinline__ float weight_of(float l, float m, float all, bool sigmoidal, bool renorm, int width,
                                           float &slope) {
    const bool some = l != -INFINITY;
    float g;
    slope = 1.f;
    if (sigmoidal) {
        g = renorm && m < 0.f ? sigmoid_over(l, m) : sigmoid(l);
        slope = sigmoid(-l);
    } else {
        g = expf(l - m);
    }
    if (!some) g = 0.f;
    if (renorm) {
        all = g;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            if (off < width) all += __shfl_xor_sync(kAll, all, off);
    } else if (sigmoidal) {
        return g;
    }
    return some ? __fdividef(g, all) : 0.f;
}

// a >= b afterwards
__device__ __forceinline__ void order2(uint32_t &a, uint32_t &b) {
    const uint32_t m = max(a, b);
    b = min(a, b);
    a = m;
}

// in falling order
__device__ __forceinline__ void sort4(uint32_t b[4]) {
    order2(b[0], b[1]);
    order2(b[2], b[3]);
    order2(b[0], b[2]);
    order2(b[1], b[3]);
    order2(b[1], b[2]);
}
// the four largest of two ordered fours, in order
__device__ __forceinline__ void merge4(uint32_t a[4], const uint32_t b[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = max(a[i], b[3 - i]);   // rising and falling
    order2(a[0], a[2]);
    order2(a[1], a[3]);
    order2(a[0], a[1]);
    order2(a[2], a[3]);
}
// two ordered fours, one behind the other, into one order
__device__ __forceinline__ void join8(uint32_t b[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) order2(b[i], b[i + 4]);
    order2(b[2], b[4]);
    order2(b[3], b[5]);
    order2(b[1], b[2]);
    order2(b[3], b[4]);
    order2(b[5], b[6]);
}
// c becomes the eight largest (rising and falling) of it and the lane's `off` away, both in order; returns the largest that is not
__device__ __forceinline__ uint32_t take8(uint32_t c[8], int off, bool count) {
    uint32_t o[8], lost = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __shfl_xor_sync(kAll, c[7 - i], off);
    if (count) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) lost = max(lost, max(min(c[i], o[i]), min(c[i + 1], o[i + 1])));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = max(c[i], o[i]);
    return lost;
}
// of eight that rise and fall
__device__ __forceinline__ void sort_bitonic8(uint32_t c[8]) {
#pragma unroll
    for (int step = 4; step >= 1; step >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & step)) order2(c[i], c[i + step]);
}
// the key that carries expert e's index
__device__ __forceinline__ uint32_t key_with(float v, int e) { return (key_of(v) & ~kIndex) | (kIndex & ~(uint32_t)e); }
// a key as choose makes them, of a choice by whole keys (e < 0: none)
__device__ __forceinline__ uint32_t key_of_choice(int e) { return e >= 0 ? ~kIndex | (kIndex - e) : 0; }

// the k largest of a row by whole keys, the expert of slot s in lane s (-1: none): each round finds the largest key of the
// warp; where several lanes hold it, the one with the lowest index wins
template <typename T, int VEC, int J>
__device__ __noinline__ int choose_exactly(const T *logits, int E, int k, int lane) {
    Row<T, VEC, J> row;
    row.load(logits, E, lane);
    uint32_t key[VEC * J];
#pragma unroll
    for (int i = 0; i < VEC * J; ++i) key[i] = key_of(row.value(i));
    int id = -1;
    for (int s = 0; s < k; ++s) {
        uint32_t best = 0;
        int at = 0;   // of this lane's largest: the lowest index
#pragma unroll
        for (int i = 0; i < VEC * J; ++i)
            if (key[i] > best) {
                best = key[i];
                at = 32 * VEC * (i / VEC) + VEC * lane + i % VEC;
            }
        const uint32_t top = __reduce_max_sync(kAll, best);
        if (top <= kNone) break;
        const int e = (int)__reduce_min_sync(kAll, best == top ? (unsigned)at : kAll);
        if (lane == s) id = e;
#pragma unroll
        for (int i = 0; i < VEC * J; ++i)
            if (32 * VEC * (i / VEC) + VEC * lane + i % VEC == e) key[i] = 0;
    }
    return id;
}

// The k + 1 largest of a row by keys that carry the index, in order, to slot[0 .. k]; true where a lane ran out of its four.
// (One more than are taken: is the last one's rank certain?)
template <typename T, int VEC, int J>
__device__ __forceinline__ bool choose(const Row<T, VEC, J> &row, int k, int lane, uint32_t *lists, uint32_t *slot) {
    uint32_t a[4] = {0, 0, 0, 0};   // the lane's largest, in order
#pragma unroll
    for (int j = 0; j < VEC * J; j += 4) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = j + i, e = 32 * VEC * (at / VEC) + VEC * lane + at % VEC;
            b[i] = at < VEC * J ? key_with(row.value(at % (VEC * J)), e) : 0;
        }
        sort4(b);
        if (j == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = b[i];
        } else {
            merge4(a, b);
        }
    }
    // The lists lie in shared memory, a lane its column, with a 0 behind them.  Whose value is the largest writes it to the
    // round's slot and takes up its next one: two instructions of the pipe that bounds this instead of eight in registers.
#pragma unroll
    for (int i = 1; i < 4; ++i) lists[32 * (i - 1) + lane] = a[i];
    uint32_t head = a[0], at = (uint32_t)__cvta_generic_to_shared(lists + lane);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot);
#pragma unroll 3
    for (int s = 0; s <= k; ++s)   // (predicated: a branch around three instructions costs as much as they do)
        asm volatile(
            "{\n .reg .pred p;\n setp.eq.u32 p, %0, %2;\n @p st.shared.u32 [%3], %2;\n @p ld.shared.u32 %0, [%1];\n"
            " @p add.u32 %1, %1, 128;\n}"
            : "+r"(head), "+r"(at) : "r"(__reduce_max_sync(kAll, head)), "r"(to + 4 * s) : "memory");
    return VEC * J > 4 && head == 0;   // (the key of an expert is not 0)
}

struct TopkArgs {
    const void *logits;
    const uint8_t *valid;
    int32_t *ids;
    float *weights;
    int T, E, k, sigmoid, renorm;
    int width, batch;   // lanes of a row's slots (a power of two), rows of a batch
};

// A warp takes a batch of rows: it makes their choices one after the other, the next row's loads under way while it works on
// one, and the weights of all of them at once, a lane a slot (a row by itself took 353 instructions at E = 256, of which
// two thirds do not depend on E).  ALL: the weights are shares of the whole row.
template <typename T, int VEC, int J, bool ALL>
__global__ void __launch_bounds__(32 * kWarps, blocks_per_sm(VEC * J)) topk_kernel(const TopkArgs a) {
    __shared__ uint32_t s_lists[kWarps][4 * 32], s_slots[kWarps][64];
    const int lane = threadIdx.x & 31, warp = blockIdx.x * kWarps + (threadIdx.x >> 5), warps = gridDim.x * kWarps;
    const int r = lane / a.width, s = lane & (a.width - 1);   // of the batch's weights
    uint32_t *lists = s_lists[threadIdx.x >> 5], *slots = s_slots[threadIdx.x >> 5];
    lists[96 + lane] = 0;
    const T *logits = static_cast<const T *>(a.logits);
    // this warp's rows: as many as any other's, but for one
    const int end = (int)((long long)a.T * (warp + 1) / warps);
    int base = (int)((long long)a.T * warp / warps);
    Row<T, VEC, J> next;
    bool next_live = false;
    const auto fetch = [&](int t) {
        if (t >= end) return;
        next_live = !a.valid || a.valid[t];
        next.load(logits + (size_t)t * a.E, a.E, lane);
    };
    fetch(base);
    for (; base < end; base += a.batch) {
        const int n = min(a.batch, end - base);
        unsigned unsure = 0;   // rows of the batch
        float all = 0.f;
        for (int i = 0; i < n; ++i) {
            const Row<T, VEC, J> row = next;
            const bool live = next_live;
            fetch(base + i + 1);
            uint32_t *slot = slots + i * (a.width + 1);
            if (live) {
                if (choose<T, VEC, J>(row, a.k, lane, lists, slot)) unsure |= 1u << i;
                if (ALL) {
                    float m = row.value(0);
#pragma unroll
                    for (int j = 1; j < VEC * J; ++j) m = max_nan(m, row.value(j));
                    const float sum = row.sum(warp_max(m));
                    if (r == i) all = sum;
                }
            } else if (lane <= a.k) {
                slot[lane] = 0;
            }
        }
        __syncwarp();
        const bool mine = r < n && s < a.k;
        const int at = min(r, n - 1) * (a.width + 1) + min(s, a.k - 1);
        uint32_t key = slots[at];
        if (sizeof(T) == 4) {
            const uint32_t below = slots[at + 1];
            if (mine && below > kNone && (key ^ below) <= kIndex) unsure |= 1u << r;
        }
        if (__any_sync(kAll, unsure)) {
            unsure = __reduce_or_sync(kAll, unsure);
            for (int i = 0; i < n; ++i) {
                if (!(unsure >> i & 1)) continue;
                const int e = choose_exactly<T, VEC, J>(logits + (size_t)(base + i) * a.E, a.E, a.k, lane);
                if (lane < a.k) slots[i * (a.width + 1) + lane] = key_of_choice(e);
            }
            __syncwarp();
            key = slots[at];
        }
        const int id = mine && key > kNone ? (int)(kIndex - (key & kIndex)) : -1;
        const float l = id >= 0 ? (float)logits[(size_t)(base + r) * a.E + id] : -INFINITY;
        const float m = __shfl_sync(kAll, l, lane - s);
        float slope;
        const float w = weight_of(l, m, all, a.sigmoid, a.renorm, a.width, slope);
        if (mine) {
            const size_t to = (size_t)(base + r) * a.k + s;
            a.ids[to] = id;
            if (a.weights) a.weights[to] = w;
        }
        __syncwarp();
    }
}

// Up to eight of up to 512, many rows: eight lanes hold a row, four rows a warp, so that four rows share what a step costs.
// Lists of a row's lanes are joined in three steps of an exchange and a merge; then all eight lanes have its eight largest.
//   - Up to 128 experts a lane orders its values down to its four largest.  What it leaves out may belong to the chosen (five of
//     eight in one lane: one row in a hundred).
//   - Above, the pieces of four values are ordered by their largest first: the eight largest values lie in the eight pieces
//     that are largest so, and each lane reads one of those again and orders its four.  This costs 3 instructions a value
//     instead of 11 (65536 x 256 in fp32: 23.6 us without it).
// `dropped`: the largest key that this lane saw left out.  In bf16 keys are exact, and so is the choice of pieces: whatever is
// left out of them is smaller than eight values, or equal with a higher index.
template <typename T, int J, bool ALL>
__global__ void __launch_bounds__(32 * kWarps, quad_blocks(J, sizeof(T))) topk_quad_kernel(const TopkArgs a) {
    constexpr int L = 8;
    const int lane = threadIdx.x & 31, s = lane & (L - 1), r = lane / L;
    const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5), warps = gridDim.x * kWarps;
    const T *logits = static_cast<const T *>(a.logits);
    const int fours = (int)(((long long)a.T + 3) / 4), end = (int)((long long)fours * (warp + 1) / warps);
    int four = (int)((long long)fours * warp / warps);
    Row<T, 4, J, L> row;
    bool next_live = false;
    if (four < end && 4 * four + r < a.T) {
        row.load(logits + (size_t)(4 * four + r) * a.E, a.E, s);
        next_live = !a.valid || a.valid[4 * four + r];
    }
    for (; four < end; ++four) {
        const int t = 4 * four + r;
        const bool live = next_live, more = four + 1 < end && t + 4 < a.T;
        float all = 0.f;
        if (ALL) {
            float m = row.value(0);
#pragma unroll
            for (int i = 1; i < 4 * J; ++i) m = max_nan(m, row.value(i));
            all = row.sum(lanes_max<L>(m));
        }
        next_live = more && (!a.valid || a.valid[t + 4]);
        const T *next = logits + (size_t)(t + 4) * a.E;
        uint32_t own[4], c[8], dropped = 0;   // the largest that this lane saw left out
        if constexpr (J <= 4) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int e = 4 * L * j + 4 * s;
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)   // (s comes below)
                    b[i] = key_with(row.v[j].value(i), 4 * L * j + i + 4 * (L - 1));
                if (more && e < a.E) row.v[j].load(next + e);   // the next row's, where these were
                sort4(b);
                if (j == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) own[i] = b[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
                        dropped = max(dropped, max(min(own[i], b[3 - i]), min(own[i + 1], b[2 - i])));
                    merge4(own, b);
                }
            }
            const uint32_t at_lane = 4 * (L - 1 - s);
            dropped |= at_lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) own[i] |= at_lane;
        } else {
#pragma unroll
            for (int j = 0; j < J; j += 8) {
                uint32_t b[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = 4 * L * (j + i) + 4 * s;
                    b[i] = key_with(largest(row.v[j + i]), 4 * L * (j + i) + 4 * (L - 1)) | (4 * (L - 1 - s));
                    if (more && e < a.E) row.v[j + i].load(next + e);
                }
                sort4(b);
                sort4(b + 4);
                join8(b);
                if (j == 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) c[i] = b[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (sizeof(T) == 4) dropped = max(dropped, min(c[i], b[7 - i]));
                        c[i] = max(c[i], b[7 - i]);
                    }
                    sort_bitonic8(c);
                }
            }
#pragma unroll
            for (int off = 1; off <= 4; off *= 2) {
                dropped = max(dropped, take8(c, off, sizeof(T) == 4));
                if (off < 4) sort_bitonic8(c);
            }
            // the eight lie the other way round in lanes 4 to 7: each lane of the row takes another one
            const int mine_at = s < 4 ? s : 7 - s;
            uint32_t mine = c[0];
#pragma unroll
            for (int i = 1; i < 4; ++i) mine = mine_at == i ? c[i] : mine;
            const int e = (int)(kIndex - (mine & kIndex));
            Raw<T, 4> v;
            if (live && mine > kNone) v.load(logits + (size_t)t * a.E + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) own[i] = live && mine > kNone ? key_with(v.value(i), e + i) : 0;
            sort4(own);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = own[i], c[7 - i] = __shfl_xor_sync(kAll, own[i], 1);
        sort_bitonic8(c);
#pragma unroll
        for (int off = 2; off <= 4; off *= 2) {
            dropped = max(dropped, take8(c, off, sizeof(T) == 4));
            sort_bitonic8(c);
        }
        uint32_t key = c[0];   // of slot s
#pragma unroll
        for (int i = 1; i < 8; ++i) key = s == i ? c[i] : key;
        // Not certain: what a lane dropped may belong to the chosen, or the last one's rank hangs on the bits that the index took.
        const uint32_t last = __shfl_sync(kAll, key, (lane & ~(L - 1)) + a.k - 1);
        bool unsure = dropped > kNone && (sizeof(T) == 4 ? dropped | kIndex : dropped) >= last, tied = false;
        if (sizeof(T) == 4) {
            const uint32_t below = __shfl_down_sync(kAll, key, 1);
            const bool close = live && s < L - 1 && s < a.k && below > kNone && (key ^ below) <= kIndex;
            unsure |= close && s == a.k - 1;
            tied = close && s < a.k - 1;   // only their order is not certain
        }
        unsigned who = __ballot_sync(kAll, unsure && live);
        for (; who; who &= ~(0xFFu << (__ffs(who) - 1 & ~(L - 1)))) {
            const int q = (__ffs(who) - 1) / L;
            const int e = choose_exactly<T, 4, (J + 3) / 4>(logits + (size_t)(4 * four + q) * a.E, a.E, a.k, lane);
            const uint32_t other = key_of_choice(__shfl_sync(kAll, e, s));
            if (r == q) key = other;
        }
        const bool mine = s < a.k && t < a.T;
        int id = mine && live && key > kNone ? (int)(kIndex - (key & kIndex)) : -1;
        float l = id >= 0 ? (float)logits[(size_t)t * a.E + id] : -INFINITY;
        if (__any_sync(kAll, tied)) {   // by whole keys (those of a choice by whole keys are in order)
            const uint32_t whole = id >= 0 ? key_of(l) : 0;
            int rank = 0, from = 0;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const uint32_t o = __shfl_sync(kAll, whole, i, L);
                const int oid = __shfl_sync(kAll, id, i, L);
                rank += o > whole || (o == whole && (id >= 0 ? oid < id : i < s));
            }
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (__shfl_sync(kAll, rank, i, L) == s) from = i;
            id = __shfl_sync(kAll, id, from, L);
            l = __shfl_sync(kAll, l, from, L);
        }
        const float m = __shfl_sync(kAll, l, lane - s);
        float slope;
        const float w = weight_of(l, m, all, a.sigmoid, a.renorm, L, slope);
        if (mine) {
            const size_t to = (size_t)t * a.k + s;
            a.ids[to] = id;
            if (a.weights) a.weights[to] = w;
        }
    }
}

struct TopkGradArgs {
    const void *logits, *addend;
    const int32_t *ids;
    const float *dweights;
    void *dlogits;
    int T, E, k, sigmoid, renorm;
};

// ROW: the gradient reaches the whole row (softmax over all E); otherwise the chosen experts.  A row takes L lanes: two or
// four rows share a warp where they fit, as most instructions do not depend on E (calls that write the same rows, 65536 of 128
// in bf16, over all E: 18.5 us with a row a warp, 12.4 with two, 11.3 with four; of 64, renormalised, 9.0 with two and 5.6
// with four).  The next row's slots and logits are under way as in topk_kernel (a row is read before it is written, by the
// warp that it belongs to: dlogits may be logits).
template <typename T, int VEC, int J, bool ROW, int L>
__global__ void __launch_bounds__(32 * kWarps, grad_blocks(VEC * J, ROW)) topk_grad_kernel(const TopkGradArgs a) {
    extern __shared__ float buf[];   // a row's values
    const int lane = threadIdx.x & (L - 1), first = (threadIdx.x & 31) / L;   // in its row; the row of the warp
    const int warp = threadIdx.x >> 5, step = gridDim.x * kWarps * (32 / L);
    float *at = buf + threadIdx.x / L * L * VEC * J;
    const T *logits = static_cast<const T *>(a.logits), *addend = static_cast<const T *>(a.addend);
    // On its way: the slots two rows ahead, and one row ahead what is read (the chosen logits need the slots).
    Row<T, VEC, J, L> next, next_add;
    int ids[2] = {-1, -1};
    float ds[2] = {}, next_mine = -INFINITY;
    const auto fetch_slots = [&](int t, int i) {
        if (t >= a.T || lane >= a.k) return;
        ids[i] = a.ids[(size_t)t * a.k + lane];
        ds[i] = a.dweights[(size_t)t * a.k + lane];
    };
    const auto fetch = [&](int t, int i) {
        if (t >= a.T) return;
        if (ROW) next.load(logits + (size_t)t * a.E, a.E, lane);
        else next_mine = (unsigned)ids[i] < (unsigned)a.E ? (float)logits[(size_t)t * a.E + ids[i]] : -INFINITY;
        if (addend) next_add.load(addend + (size_t)t * a.E, a.E, lane);
    };
    int t = (blockIdx.x * kWarps + warp) * (32 / L) + first;
    fetch_slots(t, 0);
    fetch_slots(t + step, 1);
    fetch(t, 0);
    for (; t - first < a.T; t += step) {   // (all lanes of a warp together; rows past T are not written)
        const Row<T, VEC, J, L> row = next, add = next_add;
        const int id = (unsigned)ids[0] < (unsigned)a.E && t < a.T ? ids[0] : -1;
        const float d = id >= 0 ? ds[0] : 0.f;
        float mine = next_mine;
        if (ROW) {   // from the row, through shared memory
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) at[L * VEC * j + VEC * lane + i] = row.value(VEC * j + i);
            __syncwarp();
            mine = id >= 0 ? at[id] : -INFINITY;
        }
        fetch(t + step, 1);
        ids[0] = ids[1];
        ds[0] = ds[1];
        fetch_slots(t + 2 * step, 1);
        float m = mine;
        if (ROW) {
#pragma unroll
            for (int i = 0; i < VEC * J; ++i) m = max_nan(m, row.value(i));
        }
        m = lanes_max<L>(m);
        const float all = ROW ? row.sum(m) : 0.f;
        float slope;
        const float w = weight_of(mine, m, all, a.sigmoid, a.renorm, L, slope);
        const bool ratio = a.renorm || !a.sigmoid;
        const float dot = ratio ? lanes_sum<L>(id >= 0 ? w * d : 0.f) : 0.f;
        // the row's gradient at the chosen experts; where an id comes twice (one of its slots finds the other's mark),
        // slot by slot in their order
        const float g = ROW ? w * d : slope * w * (d - dot);
        __syncwarp();
        if (id >= 0) at[id] = __int_as_float(lane);
        __syncwarp();
        const bool twice = __any_sync(kAll, id >= 0 && __float_as_int(at[id]) != lane);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) at[L * VEC * j + VEC * lane + i] = 0.f;
        __syncwarp();
        if (!twice) {
            if (id >= 0) at[id] = g;
        } else {
            for (int s = 0; s < a.k; ++s) {
                if (lane == s && id >= 0) at[id] += g;
                __syncwarp();
            }
        }
        __syncwarp();
        const float scale = ROW ? dot / all : 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = L * VEC * j + VEC * lane;
            if (e >= a.E || t >= a.T) continue;
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[i] = at[e + i];
                // a row without slots has no gradient, whatever its logits are
                if (ROW && dot != 0.f && row.value(VEC * j + i) != -INFINITY)
                    v[i] -= exp_fast(row.value(VEC * j + i) - m) * scale;
                if (addend) v[i] += add.v[j].value(i);
            }
            store_vec<T, VEC>(static_cast<T *>(a.dlogits) + (size_t)t * a.E + e, v);
        }
    }
}

unsigned blocks(int rows, int per_sm) {
    const long long need = ((long long)rows + kWarps - 1) / kWarps, most = (long long)num_sms() * per_sm;
    return (unsigned)(need < most ? need : most);
}
template <typename T, int VEC, int J>
cudaError_t topk_t(TopkArgs a, cudaStream_t s) {
    const int per_sm = blocks_per_sm(VEC * J);
    a.width = 1;
    while (a.width < a.k) a.width *= 2;
    // batches where every warp has one: few rows take the time of one
    a.batch = 32 / a.width;
    while (a.batch > 1 && (long long)num_sms() * per_sm * kWarps * a.batch > a.T) a.batch /= 2;
    const unsigned grid = blocks((a.T + a.batch - 1) / a.batch, per_sm);
    if (!a.sigmoid && !a.renorm) topk_kernel<T, VEC, J, true><<<grid, 32 * kWarps, 0, s>>>(a);
    else topk_kernel<T, VEC, J, false><<<grid, 32 * kWarps, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int J>
cudaError_t quad_t(const TopkArgs &a, cudaStream_t s) {
    const unsigned grid = blocks((int)(((long long)a.T + 3) / 4), quad_blocks(J, sizeof(T)));
    if (!a.sigmoid && !a.renorm) topk_quad_kernel<T, J, true><<<grid, 32 * kWarps, 0, s>>>(a);
    else topk_quad_kernel<T, J, false><<<grid, 32 * kWarps, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int VEC, int J, int L>
cudaError_t grad_t(const TopkGradArgs &a, cudaStream_t s) {
    constexpr int smem = kWarps * 32 * VEC * J * (int)sizeof(float);   // 32 KB at most
    const bool row = !a.sigmoid && !a.renorm;
    const unsigned grid = blocks((a.T + 32 / L - 1) / (32 / L), grad_blocks(VEC * J, row));
    if (row) topk_grad_kernel<T, VEC, J, true, L><<<grid, 32 * kWarps, smem, s>>>(a);
    else topk_grad_kernel<T, VEC, J, false, L><<<grid, 32 * kWarps, smem, s>>>(a);
    return cudaGetLastError();
}

// rows of whole 4-value pieces, or value by value
template <typename T>
cudaError_t topk_by_width(const TopkArgs &a, cudaStream_t s) {
    if (a.E % 4 == 0) {
        // (fewer rows have a warp each, with a shorter chain: 1024 x 512 take 4.3 us so, 4.7 by fours; 2048 x 512 4.9 both
        // ways, 4096 x 512 7.3 and 4.9, 1024 x 256 3.8 and 3.4)
        if (a.k <= 8 && a.E <= 512 && a.T >= 4 * a.E) {
            if (a.E <= 64) return quad_t<T, 2>(a, s);
            if (a.E <= 128) return quad_t<T, 4>(a, s);
            return a.E <= 256 ? quad_t<T, 8>(a, s) : quad_t<T, 16>(a, s);
        }
        if (a.E <= 128) return topk_t<T, 4, 1>(a, s);
        if (a.E <= 256) return topk_t<T, 4, 2>(a, s);
        if (a.E <= 512) return topk_t<T, 4, 4>(a, s);
        return topk_t<T, 4, 8>(a, s);
    }
    if (a.E <= 64) return topk_t<T, 1, 2>(a, s);
    if (a.E <= 256) return topk_t<T, 1, 8>(a, s);
    return topk_t<T, 1, 32>(a, s);
}
template <typename T>
cudaError_t grad_by_width(const TopkGradArgs &a, cudaStream_t s) {
    const bool four = a.k <= 8, two = a.k <= 16;   // rows a warp, where 8 or 16 lanes hold one
    if (a.E % 4 == 0) {
        if (a.E <= 64 && two) return four ? grad_t<T, 4, 2, 8>(a, s) : grad_t<T, 4, 1, 16>(a, s);
        if (a.E <= 128 && two) return four ? grad_t<T, 4, 4, 8>(a, s) : grad_t<T, 4, 2, 16>(a, s);
        if (a.E <= 128) return grad_t<T, 4, 1, 32>(a, s);
        if (a.E <= 256) return two ? grad_t<T, 4, 4, 16>(a, s) : grad_t<T, 4, 2, 32>(a, s);
        if (a.E <= 512) return grad_t<T, 4, 4, 32>(a, s);
        return grad_t<T, 4, 8, 32>(a, s);
    }
    if (a.E <= 64) return two ? grad_t<T, 1, 4, 16>(a, s) : grad_t<T, 1, 2, 32>(a, s);
    if (a.E <= 256) return grad_t<T, 1, 8, 32>(a, s);
    return grad_t<T, 1, 32, 32>(a, s);
}

}  // namespace

cudaError_t launch_topk(const void *logits, int dtype, const uint8_t *valid, int T, int E, int k, int gating,
                        int renormalize, int32_t *ids, float *weights, cudaStream_t s) {
    const TopkArgs a = {logits, valid, ids, weights, T, E, k, gating == MOE_GATE_SIGMOID, renormalize != 0, 0, 0};
    return dtype == MOE_DT_BF16 ? topk_by_width<__nv_bfloat16>(a, s) : topk_by_width<float>(a, s);
}

cudaError_t launch_topk_grad(const void *logits, int dtype, const int32_t *ids, const float *dweights, int T, int E,
                             int k, int gating, int renormalize, const void *addend, void *dlogits, cudaStream_t s) {
    const TopkGradArgs a = {logits, addend, ids, dweights, dlogits, T, E, k, gating == MOE_GATE_SIGMOID,
                            renormalize != 0};
    return dtype == MOE_DT_BF16 ? grad_by_width<__nv_bfloat16>(a, s) : grad_by_width<float>(a, s);
}

}  // namespace moe
