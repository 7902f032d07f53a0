// logits.hip -- log probabilities of given tokens with the entropy and the
// largest entries of rows of logits x [M][V], and their gradient.
//
// With z = x / T, c = log2(e) / T, m near the row's maximum:
//   S = sum 2^((x - m) c),  lse = ln 2 (m c + log2 S)
//   logp(v) = ln 2 ((x_v - m) c - log2 S)
//   H = ln 2 (log2 S - U / S),  U = sum 2^((x - m) c) (x - m) c
// One pass over a row keeps S and U per thread.  Rows are cut into slices where
// there are few; partial sums are then joined in the slices' order.
#include <hip/hip_runtime.h>

#include "rbq.h"
#include "rbq_kernels.h"
#include "logits_device.h"

namespace rbq {

namespace {

constexpr float LN2 = 0.6931471805599453f;

// The largest k entries of a slice, sorted, for every row whatever its values at
// a bounded cost.  Each thread knows its largest entry, and the k largest entries
// lie with the k threads whose largest entries are largest (any other has k better
// ones before it); among equal ones those whose entry comes first.  What is below
// the k-th of those maxima is dropped: of normally distributed entries about a
// tenth more than k are left.  Each of them finds its place by counting the larger
// ones.
// The vectors that hold them are known by their own largest entries, kept in LDS
// (2 bytes for 16 or 32 of the row), and only they are read again.  Where rows are
// too long for that, or too many vectors come into question (equal entries), all
// vectors of those k threads are read again: 16 bytes of a line each, which for 64
// threads costs as much as the whole row.
constexpr int LG_LEFT = 1024;       // most entries left that are placed so,
constexpr int LG_COUNTED = 256;     // and most that are counted before the k-th is looked for

template <int E, int TH>
struct lg_pick {        // (LDS)
    uint64_t list[64 * E];          // the result, 0 behind its end
    uint32_t key[TH];
    int where[TH], group[RBQ_TOP_MAX];
    uint32_t least;                 // key of the k-th thread's largest entry,
    int limit;                      // the last vector that counts where an entry equals it
    int groups, left, vectors;
    uint64_t first;
    int vector[LG_LEFT];            // vectors to read again
    union {
        uint64_t place[LG_LEFT];
        struct {
            uint64_t lists[(TH / 64) * 64 * E], waiting[(TH / 64) * 64 * E];
        };
    };
};

// Keys of one type's values, without the bits that its conversion to fp32 leaves
// equal: the search below takes a step a bit.
template <typename T>
__device__ __forceinline__ uint32_t lg_short_key(float v) {
    constexpr int SPARE = T::SPARE;
    return v > -__builtin_inff() ? lg_ordered(v) >> SPARE : 0;
}

template <int TH>
struct lg_pick<0, TH> {};

// Of 64 N keys (0: none), N a lane, one wave finds the k-th largest and, where
// several equal it, the last place (at(i) of a lane's key i, all different) that
// still belongs to the k largest.
template <int N, typename AT>
__device__ __forceinline__ void lg_find(const uint32_t (&key)[N], AT at, int k, uint32_t &least, int &limit) {
    auto count = [&](uint32_t t) __attribute__((always_inline)) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += __popcll(__ballot(key[i] >= t));
        return n;
    };
    // (a lane's two largest: 64 lanes have k keys no less than the least of the
    // lanes' largest, or second largest, which is where the search starts)
    uint32_t most = 0, second = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        second = max(second, min(most, key[i]));
        most = max(most, key[i]);
    }
    limit = 0x7FFFFFFF;
    uint32_t lo = max(1u, ~wave_max_u32_dpp(~(k <= 64 ? most : second))), hi = wave_max_u32_dpp(most) + 1;
    int above = 0;                  // keys >= hi
    if (count(lo) <= k) {           // just k, or all there are
        least = lo;
        return;
    }
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int n = count(mid);
        if (n == k) {
            least = mid;
            return;
        }
        if (n > k) {
            lo = mid;
        } else {
            hi = mid;
            above = n;
        }
    }
    // more than one has the k-th key: those of them that come first
    least = lo;
    int place[N];
    uint32_t far = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool is = key[i] == lo;
        place[i] = is ? at(i) : 0x7FFFFFFF;
        far = max(far, is ? (uint32_t)place[i] : 0u);
    }
    int no = -1, yes = (int)wave_max_u32_dpp(far);
    while (yes - no > 1) {
        const int mid = no + (yes - no) / 2;
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += __popcll(__ballot(place[i] <= mid));
        if (n >= k - above)
            yes = mid;
        else
            no = mid;
    }
    limit = yes;
}

template <typename T, int E, int TH>
__device__ __forceinline__ void lg_select(const typename T::bits *x, const lg_range &r, int k, float best, int where,
                                          const uint16_t *tops, lg_pick<E, TH> &p) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t mine = lg_short_key<T>(best);
    p.key[tid] = mine;
    p.where[tid] = where;
    if (tid == 0)
        p.groups = p.left = p.vectors = 0;
    __syncthreads();
    if (wave == 0) {
        uint32_t key[TH / 64], least;
        int limit;
#pragma unroll
        for (int i = 0; i < TH / 64; ++i)
            key[i] = p.key[i * 64 + lane];
        lg_find(key, [&](int i) __attribute__((always_inline)) { return p.where[i * 64 + lane]; }, k, least, limit);
        if (lane == 0) {
            p.least = least;
            p.limit = limit;
        }
    }
    __syncthreads();
    const uint32_t least = p.least;
    const int limit = p.limit;
    auto counts = [&](uint32_t key, int v) __attribute__((always_inline)) {
        return key > least || (key == least && v <= limit);
    };
    const int n = r.v1 - r.v0, end = min(r.v1, r.whole);
    // the entries of vector v that count (every lane of a wave takes part)
    auto offer = [&](int v, const float(&e)[LG_VEC], auto take) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < LG_VEC; ++j)
            take(lg_key(e[j], v * LG_VEC + j), counts(lg_short_key<T>(e[j]), v));
    };
    auto keep = [&](uint64_t key, bool is) __attribute__((always_inline)) {
        if (is) {
            const int i = atomicAdd(&p.left, 1);
            if (i < LG_LEFT)
                p.place[i] = key;
        }
    };
    if (tops != nullptr) {
        const uint32_t bound = (least << T::SPARE) >> 16;
        for (int i = tid * 8; i < n; i += TH * 8) {
            const uint4 w = *(const uint4 *)(tops + i);
            const uint32_t h[8] = {w.x & 0xFFFF, w.x >> 16, w.y & 0xFFFF, w.y >> 16,
                                   w.z & 0xFFFF, w.z >> 16, w.w & 0xFFFF, w.w >> 16};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (h[j] >= bound && i + j < n) {
                    const int at = atomicAdd(&p.vectors, 1);
                    if (at < LG_LEFT)
                        p.vector[at] = r.v0 + i + j;
                }
        }
    }
    const bool look = counts(mine, where);
    if (look)
        p.group[atomicAdd(&p.groups, 1)] = tid;
    __syncthreads();
    const int vectors = p.vectors;
    const bool known = tops != nullptr && vectors <= LG_LEFT;
    if (known) {
        for (int i = tid; i < vectors; i += TH) {
            const int v = p.vector[i];
            float e[LG_VEC];
            if (v < end)
                lg_values<T>(lg_load<T>(x + (int64_t)v * LG_VEC), e);
            else
                lg_load_part<T>(x + (int64_t)v * LG_VEC, r.rest, e);
            offer(v, e, keep);
        }
    }
    const int groups = p.groups, turns = (n + TH - 1) / TH;
    // take(key, whether it counts) of those threads' entries; every lane of a wave
    // takes part each time
    constexpr int AHEAD = 4;
    auto again = [&](auto take) __attribute__((always_inline)) {
        const int items = groups * turns;
        for (int q0 = wave * 64; q0 < items; q0 += AHEAD * TH) {
            typename T::raw raw[AHEAD];
            int v[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int q = q0 + i * TH + lane;
                v[i] = q < items ? r.v0 + p.group[q / turns] + q % turns * TH : r.v1;
                if (v[i] < end)
                    raw[i] = lg_load<T>(x + (int64_t)v[i] * LG_VEC);
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                float e[LG_VEC];
                if (v[i] < end) {
                    lg_values<T>(raw[i], e);
                } else {
                    const int n = v[i] < r.v1 ? r.rest : 0;
                    lg_load_part<T>(x + (int64_t)v[i] * LG_VEC, n, e);
                }
                offer(v[i], e, take);
            }
        }
    };
    if (!known)
        again(keep);
    __syncthreads();
    const int left = p.left;
    if (left <= LG_LEFT) {
        int ranked = left;
        uint64_t first = 1;     // the least key that counts
        if (left > LG_COUNTED) {
            // too many to count: the k-th largest is looked for first
            if (wave == 0) {
                uint32_t key[LG_LEFT / 64], kth;
                int last;
#pragma unroll
                for (int i = 0; i < LG_LEFT / 64; ++i)
                    key[i] = i * 64 + lane < left ? (uint32_t)(p.place[i * 64 + lane] >> 32) : 0;
                lg_find(key, [&](int i) __attribute__((always_inline)) { return lg_index(p.place[i * 64 + lane]); }, k, kth, last);
                if (lane == 0)
                    p.first = (uint64_t)kth << 32 | (uint32_t)~last;
            }
            __syncthreads();
            first = p.first;
        }
        // (behind the end: keys of no entry, up to whole eights)
        if (tid < -left % 8 + 8 && left + tid < LG_LEFT)
            p.place[left + tid] = 0;
        __syncthreads();
        if (left > LG_COUNTED) {
            // those that count, moved together
            uint64_t mine[LG_LEFT / TH];
#pragma unroll
            for (int i = 0; i < LG_LEFT / TH; ++i)
                mine[i] = i * TH + tid < left ? p.place[i * TH + tid] : 0;
            if (tid == 0)
                p.left = 0;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < LG_LEFT / TH; ++i)
                if (mine[i] >= first)
                    p.place[atomicAdd(&p.left, 1)] = mine[i];
            __syncthreads();
            ranked = p.left;
            if (tid < -ranked % 8 + 8)
                p.place[ranked + tid] = 0;
            __syncthreads();
        }
        for (int i = tid; i < ranked; i += TH) {
            const uint64_t key = p.place[i];
            int larger = 0;
            for (int j = 0; j < ranked; j += 8)
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    larger += p.place[j + h] > key;
            if (larger < k)
                p.list[larger] = key;
        }
        for (int j = left + tid; j < k; j += TH)
            p.list[j] = 0;
    } else {        // rows made for it (many entries above the k-th maximum with few threads)
        lg_top<E> top;
        top.start(p.waiting + wave * 64 * E);
        again([&](uint64_t key, bool is) __attribute__((always_inline)) { top.offer(key, is); });
        top.settle();
        lg_block_merge<E, TH / 64>(top.k, p.lists);
        for (int j = tid; j < k; j += TH)
            p.list[j] = p.lists[j];
    }
    __syncthreads();
}

struct lg_logp_args {
    const int64_t *targets;
    float *logp, *entropy, *top_logp;
    int32_t *top_index;
    int top;
    const float *d_logp, *d_entropy;
    void *dx;
    int64_t d_stride;
};

// A row's sums and what follows from them.
struct lg_logp_row : lg_row {
    float logS, H;          // log2 S; entropy in nats
    bool empty;             // no entry above -inf
    __device__ __forceinline__ lg_logp_row(const lg_row &r) : lg_row(r) {
        empty = S == 0.0f;
        logS = log2f(S);
        H = empty ? 0.0f : fmaxf(logS - b / S, 0.0f) * LN2;
        if (S != S)
            H = S;
    }
    // (The lowest values a mask may use have infinite exponents, and log
    // probabilities that are finite.)
    __device__ __forceinline__ float logp(float v, float c, float inv_t) const {
        const float d = exponent(v, c);
        return d >= LG_LOWEST ? (d - logS) * LN2 : quick ? v * inv_t : __builtin_fmaf(-LN2, logS, (v - m) * inv_t);
    }
};

// The log probability of a row's target with logit v: 0 for none (negative), NaN
// for one beyond the vocabulary.
__device__ __forceinline__ float lg_target(const lg_logp_row &r, float v, int64_t target, const lg_row_args &a) {
    if (target < 0)
        return 0.0f;
    if (target >= a.V)
        return __builtin_nanf("");
    return r.empty ? -__builtin_inff() : r.logp(v, a.c, a.inv_t);
}

// A row's token beyond the vocabulary is reported whatever is asked of the row.
__device__ __forceinline__ void lg_report(int64_t target, const lg_row_args &a) {
    if (target >= a.V && a.status != nullptr)
        atomicOr(a.status, RBQ_STATUS_BAD_TOKEN);
}

// What thread 0 writes of a row.  The target's logit is found in the row, or,
// where rows are cut, beside the sums of the slice that holds it: x may be the
// gradient's buffer, which other slices' workgroups are writing by then.
__device__ __forceinline__ void lg_write_logp(const lg_logp_row &r, float v, int64_t target, int row, const lg_row_args &a,
                                              const lg_logp_args &p) {
    if (p.logp != nullptr)
        p.logp[row] = lg_target(r, v, target, a);
    if (p.entropy != nullptr)
        p.entropy[row] = r.H;
}
__device__ __forceinline__ bool lg_inside(int64_t target, int V) { return target >= 0 && target < V; }
__device__ __forceinline__ float lg_kept(const float4 *part, int64_t target, const lg_row_args &a) {
    return lg_inside(target, a.V) ? part[(int)target / LG_VEC / lg_each(a.V, a.slices)].w : 0.0f;
}

__device__ __forceinline__ void lg_write_top(const lg_logp_row &r, const uint64_t *list, int row, float c, float inv_t,
                                             const lg_logp_args &p) {
    for (int j = threadIdx.x; j < p.top; j += blockDim.x) {
        const uint64_t key = list[j];
        const bool broken = r.S != r.S;
        p.top_logp[(int64_t)row * p.top + j] = broken   ? r.S
                                               : key == 0 ? -__builtin_inff()
                                                          : r.logp(lg_value(key), c, inv_t);
        p.top_index[(int64_t)row * p.top + j] = broken || key == 0 ? -1 : lg_index(key);
    }
}

// The sums of a whole row: quickly, and once more where that was not good.
template <typename T, bool TOP, int TH>
__device__ __forceinline__ lg_row lg_whole_row(lg_walk<T, TH> &walk, float c, float4 *part, float &best, int &where,
                                               uint16_t *tops) {
    {
        lg_sums<true> s;
        lg_stream<T, LG_ENTROPY, TOP>(walk, c, nullptr, 0, s, best, where, tops);
        const lg_sums<true> t = lg_join_block<LG_ENTROPY, TH>(s, c, part);
        if (lg_good(t))
            return lg_row_of(t);
    }
    __syncthreads();
    lg_sums<false> s;
    float b2;
    int w2;
    lg_stream<T, LG_ENTROPY, false>(walk, c, nullptr, 0, s, b2, w2);
    return lg_row_of(lg_join_block<LG_ENTROPY, TH>(s, c, part));
}

// The sums of a slice per workgroup (SLICED), or a whole row, and its largest
// entries.  E = 0: none.  One read of the logits bounds it: 2048 x 128256 fp16, 97 us
// alone (5.4 TB/s; a plain read 5.8), 110 with 64 alternatives, whose search reads the
// vectors that can hold them again.  One row of 32000 with 20: 11 us on the device,
// the steps of the search (5.2 without).
template <typename T, int E, int TH, bool SLICED>
__global__ __launch_bounds__(TH) void logprobs_kernel(lg_row_args a, lg_logp_args p) {
    __shared__ float4 part[(TH / 64)];
    __shared__ lg_pick<E, TH> pick;
    extern __shared__ __align__(16) uint16_t vector_tops[];
    uint16_t *tops = E > 0 && lg_each(a.V, a.slices) <= LG_TOPS ? vector_tops : nullptr;
    const int64_t u = a.first + blockIdx.x;
    const int row = (int)(u / a.slices), slice = (int)(u - (int64_t)row * a.slices);
    const typename T::bits *x = (const typename T::bits *)a.x + row * a.stride;
    const lg_range r = lg_slice(a.V, a.slices, slice);
    const int64_t target = p.targets == nullptr ? -1 : p.targets[row];
    if (slice == 0 && threadIdx.x == 0)
        lg_report(target, a);
    float best = -__builtin_inff();
    int where = 0;
    lg_walk<T, TH> walk(x, r);
    lg_row sums;
    if constexpr (SLICED) {
        lg_sums<false> s;
        lg_stream<T, LG_ENTROPY, (E > 0)>(walk, a.c, nullptr, r.v0, s, best, where, tops);
        sums = lg_row_of(lg_join_block<LG_ENTROPY, TH>(s, a.c, part));
    } else {
        sums = lg_whole_row<T, (E > 0)>(walk, a.c, part, best, where, tops);
    }
    if constexpr (E > 0)
        lg_select<T, E, TH>(x, r, p.top, best, where, tops, pick);
    if constexpr (SLICED) {
        if (threadIdx.x == 0) {
            const bool here = lg_inside(target, a.V) && target >= (int64_t)r.v0 * LG_VEC &&
                              target < (int64_t)r.v1 * LG_VEC;
            a.sums[u] = make_float4(sums.m, sums.S, sums.b, here ? T::one(x[target]) : 0.0f);
        }
        if constexpr (E > 0)
            for (int j = threadIdx.x; j < p.top; j += TH)
                a.keys[u * p.top + j] = pick.list[j];
    } else {
        const lg_logp_row w(sums);
        if (threadIdx.x == 0)
            lg_write_logp(w, lg_inside(target, a.V) ? T::one(x[target]) : 0.0f, target, row, a, p);
        if constexpr (E > 0)
            lg_write_top(w, pick.list, row, a.c, a.inv_t, p);
    }
}

// The slices of a row joined.
constexpr int LG_JOIN = 512;

template <int E>
__global__ __launch_bounds__(LG_JOIN) void logprobs_join_kernel(lg_row_args a, lg_logp_args p) {
    constexpr int N = (LG_JOIN / 64) * 64 * (E > 0 ? E : 1);
    __shared__ float4 part[LG_SLICES_MAX];
    __shared__ uint64_t lists[E > 0 ? N : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = (int)(a.first + blockIdx.x);
    for (int i = threadIdx.x; i < a.slices; i += LG_JOIN)
        part[i] = a.sums[(int64_t)row * a.slices + i];
    if constexpr (E > 0) {
        uint64_t best[E], next[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            best[e] = 0;
        for (int i = wave; i < a.slices; i += (LG_JOIN / 64)) {
            const uint64_t *list = a.keys + ((int64_t)row * a.slices + i) * p.top;
            lg_wave_sync();
#pragma unroll
            for (int e = 0; e < E; ++e) {
                next[e] = e * 64 + lane < p.top ? list[e * 64 + lane] : 0;
                lists[wave * 64 * E + e * 64 + lane] = next[e];
            }
            lg_wave_sync();
            lg_merge<E>(best, lists + wave * 64 * E);
        }
        __syncthreads();
        lg_block_merge<E, LG_JOIN / 64>(best, lists);
    }
    __syncthreads();
    const lg_logp_row w(lg_row_of(lg_join_list<LG_ENTROPY, false>(part, a.slices, a.c)));
    if (threadIdx.x == 0) {
        const int64_t target = p.targets == nullptr ? -1 : p.targets[row];
        lg_write_logp(w, lg_kept(part, target, a), target, row, a, p);
    }
    if constexpr (E > 0)
        lg_write_top(w, lists, row, a.c, a.inv_t, p);
}

// The gradient of sum_m a_m logp_m + b_m H_m:
//   dx_v = (a ([v = target] - p_v) - b p_v (ln p_v + H)) / T
// with p_v = e_v / S and ln p_v = ln 2 (d_v - log2 S), so that the part without
// the target is e_v (w0 + w1 d_v).  Where rows are whole the sums are formed here,
// and the second pass over the row finds it in the caches.
template <typename T, bool QUICK, bool ENTROPY, int TH>
__device__ __forceinline__ void lg_logp_grad(lg_walk<T, TH> &walk, typename T::bits *dx, float m, float c, float w0,
                                             float w1, int at, int in, float own) {
    walk.down(dx, [&](float(&e)[LG_VEC], int v) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LG_VEC; ++i) {
            const float d = lg_exponent<QUICK>(e[i], m, c);
            const float g = __builtin_amdgcn_exp2f(d);
            e[i] = ENTROPY ? g * __builtin_fmaf(w1, fmaxf(d, LG_FAR), w0) : g * w0;
        }
        if (v == at) {
#pragma unroll
            for (int i = 0; i < LG_VEC; ++i)
                e[i] += i == in ? own : 0.0f;
        }
    });
}

// The row's sums, then a second walk from its end, whose last vectors are still in the
// cache or in LDS, that writes the gradient past it.  Bound by the read and the write:
// 2048 x 32000 fp16 52 to 55 us (5.0 TB/s of both, a copy 5.2), 2048 x 128256 237 (4.4),
// 333 x 50257 bf16 with the entropy's part 21.6 (3.1: 333 workgroups on 256 CUs).
template <typename T, int TH, bool SLICED, bool ENTROPY>
__global__ __launch_bounds__(TH) void logprobs_grad_kernel(lg_row_args a, lg_logp_args p) {
    __shared__ float4 part[SLICED ? LG_SLICES_MAX : TH / 64];
    const int64_t u = a.first + blockIdx.x;
    const int row = (int)(u / a.slices), slice = (int)(u - (int64_t)row * a.slices);
    const typename T::bits *x = (const typename T::bits *)a.x + row * a.stride;
    typename T::bits *dx = (typename T::bits *)p.dx + row * p.d_stride;
    const lg_range r = lg_slice(a.V, a.slices, slice);
    const int64_t target = p.targets == nullptr ? -1 : p.targets[row];
    const float wa = p.d_logp == nullptr || target < 0 ? 0.0f : p.d_logp[row];
    const float wb = ENTROPY ? p.d_entropy[row] : 0.0f;
    if (!SLICED && threadIdx.x == 0)
        lg_report(target, a);       // (cut rows: with their sums)
    const bool none = wa == 0.0f && wb == 0.0f;
    if (none && p.logp == nullptr && p.entropy == nullptr) {
        lg_zero<T, TH>(dx, r);
        return;
    }
    __shared__ uint4 held[SLICED ? 1 : lg_walk<T, TH>::HELD_BYTES / 16];
    // (few rows stay in the caches: 333 x 50257 bf16 21.6 us without, 24.1 held; 512 x
    // 32000 fp16 16.6 and 16.3)
    lg_walk<T, TH> walk(x, r, SLICED || a.M < 512 ? nullptr : held);
    lg_row sums;
    if constexpr (SLICED) {
        for (int i = threadIdx.x; i < a.slices; i += TH)
            part[i] = a.sums[(int64_t)row * a.slices + i];
        __syncthreads();
        sums = lg_row_of(lg_join_list<LG_ENTROPY, false>(part, a.slices, a.c));
    } else {
        float best;
        int where;
        sums = lg_whole_row<T, false>(walk, a.c, part, best, where, nullptr);
    }
    const lg_logp_row w(sums);
    if (slice == 0 && threadIdx.x == 0)
        lg_write_logp(w,
                      SLICED                      ? lg_kept(part, target, a)
                      : lg_inside(target, a.V) ? T::one(x[target])
                                                 : 0.0f,
                      target, row, a, p);
    __syncthreads();    // the target's entry has been read: dx may be x, of rows without weight too
    // (the entropy's part does not depend on the token)
    const bool bad = target >= a.V && wa != 0.0f;
    if (none || (w.empty && !bad)) {
        lg_zero<T, TH>(dx, r);
    } else {
        const float scale = a.inv_t / w.S;
        const float w0 = bad ? __builtin_nanf("") : -scale * (wa + wb * (w.H - LN2 * w.logS)), w1 = -scale * wb * LN2;
        const int at = lg_inside(target, a.V) ? (int)target / LG_VEC : -1, in = (int)target % LG_VEC;
        const float own = wa * a.inv_t;
        if (!SLICED && w.quick)
            lg_logp_grad<T, true, ENTROPY>(walk, dx, w.m, a.c, w0, w1, at, in, own);
        else
            lg_logp_grad<T, false, ENTROPY>(walk, dx, w.m, a.c, w0, w1, at, in, own);
    }
}

// f(threads of a workgroup) for a slice of `each` vectors and k alternatives.
template <typename F>
void with_threads(int each, int k, F f) {
    const int n = logits_threads(each, k);
    if (n == 512)
        f(std::integral_constant<int, 512>{});
    else if (n == 256)
        f(std::integral_constant<int, 256>{});
    else
        f(std::integral_constant<int, 128>{});
}

template <typename T>
hipError_t logprobs_of(lg_row_args a, const lg_logp_args &p, hipStream_t st) {
    const int64_t units = (int64_t)a.M * a.slices;
    const int each = lg_each(a.V, a.slices);
    auto run = [&](auto e, auto th) {
        constexpr int E = decltype(e)::value, TH = decltype(th)::value;
        const size_t tops = E > 0 && each <= LG_TOPS ? ((size_t)each * 2 + 15) / 16 * 16 : 0;
        if (a.slices > 1) {
            lg_launches(a, units, [&](unsigned n) { logprobs_kernel<T, E, TH, true><<<n, TH, tops, st>>>(a, p); });
            lg_launches(a, a.M, [&](unsigned n) { logprobs_join_kernel<E><<<n, LG_JOIN, 0, st>>>(a, p); });
        } else {
            lg_launches(a, units, [&](unsigned n) { logprobs_kernel<T, E, TH, false><<<n, TH, tops, st>>>(a, p); });
        }
    };
    with_threads(each, p.top, [&](auto th) {
        if (p.top == 0)
            run(std::integral_constant<int, 0>{}, th);
        else if (p.top <= 64)
            run(std::integral_constant<int, 1>{}, th);
        else if constexpr (decltype(th)::value > 128)
            run(std::integral_constant<int, 2>{}, th);
    });
    return hipGetLastError();
}

template <typename T, bool ENTROPY>
hipError_t logprobs_grad_of(lg_row_args a, const lg_logp_args &p, hipStream_t st) {
    const int64_t units = (int64_t)a.M * a.slices;
    with_threads(lg_each(a.V, a.slices), 0, [&](auto th) {
        constexpr int TH = decltype(th)::value;
        if (a.slices > 1) {
            lg_launches(a, units, [&](unsigned n) { logprobs_kernel<T, 0, TH, true><<<n, TH, 0, st>>>(a, p); });
            lg_launches(a, units, [&](unsigned n) { logprobs_grad_kernel<T, TH, true, ENTROPY><<<n, TH, 0, st>>>(a, p); });
        } else {
            lg_launches(a, units, [&](unsigned n) { logprobs_grad_kernel<T, TH, false, ENTROPY><<<n, TH, 0, st>>>(a, p); });
        }
    });
    return hipGetLastError();
}

template <typename T>
hipError_t logprobs_grad_any(const lg_row_args &a, const lg_logp_args &p, hipStream_t st) {
    return p.d_entropy != nullptr ? logprobs_grad_of<T, true>(a, p, st) : logprobs_grad_of<T, false>(a, p, st);
}

}  // namespace

hipError_t launch_token_logprobs(const void *x, uint32_t type, int M, int V, int64_t stride, float temperature,
                                 const int64_t *targets, float *logp, float *entropy, int top, float *top_logp,
                                 int32_t *top_index, void *workspace, size_t bytes, int32_t *status, hipStream_t st) {
    lg_row_args a = row_args(x, M, V, stride, temperature, status);
    lg_logp_args p = {};
    p.targets = targets;
    p.logp = logp;
    p.entropy = entropy;
    p.top = top;
    p.top_logp = top_logp;
    p.top_index = top_index;
    cut_rows(a, top, 0, workspace, bytes);
    return type == RBQ_L_F16   ? logprobs_of<lg_f16>(a, p, st)
           : type == RBQ_L_F32 ? logprobs_of<lg_f32>(a, p, st)
                               : logprobs_of<lg_bf16>(a, p, st);
}

hipError_t launch_token_logprobs_backward(const void *x, uint32_t type, int M, int V, int64_t stride,
                                          float temperature, const int64_t *targets, const float *d_logp,
                                          const float *d_entropy, void *dx, int64_t d_stride, float *logp,
                                          float *entropy, void *workspace, size_t bytes, int32_t *status,
                                          hipStream_t st) {
    lg_row_args a = row_args(x, M, V, stride, temperature, status);
    lg_logp_args p = {};
    p.targets = targets;
    p.logp = logp;
    p.entropy = entropy;
    p.d_logp = d_logp;
    p.d_entropy = d_entropy;
    p.dx = dx;
    p.d_stride = d_stride;
    cut_rows(a, 0, 0, workspace, bytes);
    return type == RBQ_L_F16   ? logprobs_grad_any<lg_f16>(a, p, st)
           : type == RBQ_L_F32 ? logprobs_grad_any<lg_f32>(a, p, st)
                               : logprobs_grad_any<lg_bf16>(a, p, st);
}

}  // namespace rbq
