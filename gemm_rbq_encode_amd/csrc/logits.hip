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
constexpr int LG_LEFT = 1024;       // entries left that are placed by counting

template <int E>
struct lg_pick {        // (LDS)
    uint64_t list[64 * E];          // the result, 0 behind its end
    uint32_t key[LG_THREADS];
    int where[LG_THREADS], group[RBQ_TOP_MAX];
    uint32_t least;                 // key of the k-th thread's largest entry,
    int limit;                      // the last vector that counts where an entry equals it
    int groups, left, vectors;
    int vector[LG_LEFT];            // vectors to read again
    union {
        uint64_t place[LG_LEFT];
        struct {
            uint64_t lists[LG_WAVES * 64 * E], waiting[LG_WAVES * 64 * E];
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

template <>
struct lg_pick<0> {};

// One wave finds the least key and the limit.
__device__ __forceinline__ void lg_find(const uint32_t *keys, const int *where, int k, uint32_t &least, int &limit) {
    constexpr int N = LG_THREADS / 64;
    const int lane = threadIdx.x & 63;
    // (a lane's two largest: 64 lanes have k entries no less than the least of the
    // lanes' largest, or second largest, which is where the search starts)
    uint32_t key[N], most = 0, second = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        key[i] = keys[i * 64 + lane];
        second = max(second, min(most, key[i]));
        most = max(most, key[i]);
    }
    auto count = [&](uint32_t t) __attribute__((always_inline)) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += __popcll(__ballot(key[i] >= t));
        return n;
    };
    limit = 0x7FFFFFFF;
    uint32_t lo = max(1u, ~wave_max_u32_dpp(~(k <= 64 ? most : second))), hi = wave_max_u32_dpp(most) + 1;
    int above = 0;                  // keys >= hi
    if (count(lo) <= k) {           // just k, or every thread with an entry
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
    // more than one thread has the k-th key: those of them that come first
    least = lo;
    int at[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        at[i] = key[i] == lo ? where[i * 64 + lane] : 0x7FFFFFFF;
    int no = -1, yes = 0x7FFFFFFE;
    while (yes - no > 1) {
        const int mid = no + (yes - no) / 2;
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += __popcll(__ballot(at[i] <= mid));
        if (n >= k - above)
            yes = mid;
        else
            no = mid;
    }
    limit = yes;
}

template <typename T, int E>
__device__ __forceinline__ void lg_select(const typename T::bits *x, const lg_range &r, int k, float best, int where,
                                          const uint16_t *tops, lg_pick<E> &p) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t mine = lg_short_key<T>(best);
    p.key[tid] = mine;
    p.where[tid] = where;
    if (tid == 0)
        p.groups = p.left = p.vectors = 0;
    __syncthreads();
    if (wave == 0) {
        uint32_t least;
        int limit;
        lg_find(p.key, p.where, k, least, limit);
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
        for (int i = tid * 8; i < n; i += LG_THREADS * 8) {
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
        for (int i = tid; i < vectors; i += LG_THREADS) {
            const int v = p.vector[i];
            float e[LG_VEC];
            if (v < end)
                lg_values<T>(lg_load<T>(x + (int64_t)v * LG_VEC), e);
            else
                lg_load_part<T>(x + (int64_t)v * LG_VEC, r.rest, e);
            offer(v, e, keep);
        }
    }
    const int groups = p.groups, turns = (n + LG_THREADS - 1) / LG_THREADS;
    // take(key, whether it counts) of those threads' entries; every lane of a wave
    // takes part each time
    constexpr int AHEAD = 4;
    auto again = [&](auto take) __attribute__((always_inline)) {
        const int items = groups * turns;
        for (int q0 = wave * 64; q0 < items; q0 += AHEAD * LG_THREADS) {
            typename T::raw raw[AHEAD];
            int v[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int q = q0 + i * LG_THREADS + lane;
                v[i] = q < items ? r.v0 + p.group[q / turns] + q % turns * LG_THREADS : r.v1;
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
        // (behind the end: keys of no entry, up to whole eights)
        if (tid < -left % 8 + 8 && left + tid < LG_LEFT)
            p.place[left + tid] = 0;
        __syncthreads();
        for (int i = tid; i < left; i += LG_THREADS) {
            const uint64_t key = p.place[i];
            int larger = 0;
            for (int j = 0; j < left; j += 8)
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    larger += p.place[j + h] > key;
            if (larger < k)
                p.list[larger] = key;
        }
        for (int j = left + tid; j < k; j += LG_THREADS)
            p.list[j] = 0;
    } else {        // rows made for it (many entries above the k-th maximum with few threads)
        lg_top<E> top;
        top.start(p.waiting + wave * 64 * E);
        again([&](uint64_t key, bool is) __attribute__((always_inline)) { top.offer(key, is); });
        top.settle();
        lg_block_merge<E, LG_WAVES>(top.k, p.lists);
        for (int j = tid; j < k; j += LG_THREADS)
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
    if (target >= a.V) {
        if (a.status != nullptr)
            atomicOr(a.status, RBQ_STATUS_BAD_TOKEN);
        return __builtin_nanf("");
    }
    return r.empty ? -__builtin_inff() : r.logp(v, a.c, a.inv_t);
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
template <typename T, bool TOP>
__device__ __forceinline__ lg_row lg_whole_row(lg_walk<T> &walk, float c, float4 *part, float &best, int &where,
                                               uint16_t *tops) {
    {
        lg_sums<true> s;
        lg_stream<T, LG_ENTROPY, TOP>(walk, c, nullptr, 0, s, best, where, tops);
        const lg_sums<true> t = lg_join_block<LG_ENTROPY>(s, c, part);
        if (lg_good(t))
            return lg_row_of(t);
    }
    __syncthreads();
    lg_sums<false> s;
    float b2;
    int w2;
    lg_stream<T, LG_ENTROPY, false>(walk, c, nullptr, 0, s, b2, w2);
    return lg_row_of(lg_join_block<LG_ENTROPY>(s, c, part));
}

// The sums of a slice per workgroup (SLICED), or a whole row, and its largest
// entries.  E = 0: none.
template <typename T, int E, bool SLICED>
__global__ __launch_bounds__(LG_THREADS) void logprobs_kernel(lg_row_args a, lg_logp_args p) {
    __shared__ float4 part[LG_WAVES];
    __shared__ lg_pick<E> pick;
    extern __shared__ __align__(16) uint16_t vector_tops[];
    uint16_t *tops = E > 0 && lg_each(a.V, a.slices) <= LG_TOPS ? vector_tops : nullptr;
    const int64_t u = a.first + blockIdx.x;
    const int row = (int)(u / a.slices), slice = (int)(u - (int64_t)row * a.slices);
    const typename T::bits *x = (const typename T::bits *)a.x + row * a.stride;
    const lg_range r = lg_slice(a.V, a.slices, slice);
    const int64_t target = p.targets == nullptr ? -1 : p.targets[row];
    float best = -__builtin_inff();
    int where = 0;
    lg_walk<T> walk(x, r);
    lg_row sums;
    if constexpr (SLICED) {
        lg_sums<false> s;
        lg_stream<T, LG_ENTROPY, (E > 0)>(walk, a.c, nullptr, r.v0, s, best, where, tops);
        sums = lg_row_of(lg_join_block<LG_ENTROPY>(s, a.c, part));
    } else {
        sums = lg_whole_row<T, (E > 0)>(walk, a.c, part, best, where, tops);
    }
    if constexpr (E > 0)
        lg_select<T, E>(x, r, p.top, best, where, tops, pick);
    if constexpr (SLICED) {
        if (threadIdx.x == 0) {
            const bool here = lg_inside(target, a.V) && target >= (int64_t)r.v0 * LG_VEC &&
                              target < (int64_t)r.v1 * LG_VEC;
            a.sums[u] = make_float4(sums.m, sums.S, sums.b, here ? T::one(x[target]) : 0.0f);
        }
        if constexpr (E > 0)
            for (int j = threadIdx.x; j < p.top; j += LG_THREADS)
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
template <int E>
__global__ __launch_bounds__(LG_THREADS) void logprobs_join_kernel(lg_row_args a, lg_logp_args p) {
    constexpr int N = LG_WAVES * 64 * (E > 0 ? E : 1);
    __shared__ float4 part[LG_SLICES_MAX];
    __shared__ uint64_t lists[E > 0 ? N : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = (int)(a.first + blockIdx.x);
    for (int i = threadIdx.x; i < a.slices; i += LG_THREADS)
        part[i] = a.sums[(int64_t)row * a.slices + i];
    if constexpr (E > 0) {
        uint64_t best[E], next[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            best[e] = 0;
        for (int i = wave; i < a.slices; i += LG_WAVES) {
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
        lg_block_merge<E, LG_WAVES>(best, lists);
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
template <typename T, bool QUICK, bool ENTROPY>
__device__ __forceinline__ void lg_logp_grad(lg_walk<T> &walk, typename T::bits *dx, float m, float c, float w0,
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

template <typename T, bool SLICED, bool ENTROPY>
__global__ __launch_bounds__(LG_THREADS) void logprobs_grad_kernel(lg_row_args a, lg_logp_args p) {
    __shared__ float4 part[LG_SLICES_MAX];
    const int64_t u = a.first + blockIdx.x;
    const int row = (int)(u / a.slices), slice = (int)(u - (int64_t)row * a.slices);
    const typename T::bits *x = (const typename T::bits *)a.x + row * a.stride;
    typename T::bits *dx = (typename T::bits *)p.dx + row * p.d_stride;
    const lg_range r = lg_slice(a.V, a.slices, slice);
    const int64_t target = p.targets == nullptr ? -1 : p.targets[row];
    const float wa = p.d_logp == nullptr || target < 0 ? 0.0f : p.d_logp[row];
    const float wb = ENTROPY ? p.d_entropy[row] : 0.0f;
    const bool none = wa == 0.0f && wb == 0.0f;
    if (none && p.logp == nullptr && p.entropy == nullptr) {
        lg_zero<T>(dx, r);
        return;
    }
    lg_walk<T> walk(x, r);
    lg_row sums;
    if constexpr (SLICED) {
        for (int i = threadIdx.x; i < a.slices; i += LG_THREADS)
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
    if (none || w.empty) {
        lg_zero<T>(dx, r);
    } else {
        const float scale = a.inv_t / w.S;
        const float bad = target >= a.V ? __builtin_nanf("") : 0.0f;
        const float w0 = -scale * (wa + wb * (w.H - LN2 * w.logS)) + bad, w1 = -scale * wb * LN2;
        const int at = target < 0 ? -1 : (int)(target / LG_VEC), in = (int)(target % LG_VEC);
        const float own = wa * a.inv_t;
        __syncthreads();    // the target's entry has been read: dx may be x
        if (!SLICED && w.quick)
            lg_logp_grad<T, true, ENTROPY>(walk, dx, w.m, a.c, w0, w1, at, in, own);
        else
            lg_logp_grad<T, false, ENTROPY>(walk, dx, w.m, a.c, w0, w1, at, in, own);
    }
    __syncthreads();
}

template <typename T>
hipError_t logprobs_of(lg_row_args a, const lg_logp_args &p, hipStream_t st) {
    const int64_t units = (int64_t)a.M * a.slices;
    auto run = [&](auto e) {
        constexpr int E = decltype(e)::value;
        const int each = lg_each(a.V, a.slices);
        const size_t tops = E > 0 && each <= LG_TOPS ? ((size_t)each * 2 + 15) / 16 * 16 : 0;
        if (a.slices > 1) {
            lg_launches(a, units, [&](unsigned n) { logprobs_kernel<T, E, true><<<n, LG_THREADS, tops, st>>>(a, p); });
            lg_launches(a, a.M, [&](unsigned n) { logprobs_join_kernel<E><<<n, LG_THREADS, 0, st>>>(a, p); });
        } else {
            lg_launches(a, units, [&](unsigned n) { logprobs_kernel<T, E, false><<<n, LG_THREADS, tops, st>>>(a, p); });
        }
    };
    if (p.top == 0)
        run(std::integral_constant<int, 0>{});
    else if (p.top <= 64)
        run(std::integral_constant<int, 1>{});
    else
        run(std::integral_constant<int, 2>{});
    return hipGetLastError();
}

template <typename T, bool ENTROPY>
hipError_t logprobs_grad_of(lg_row_args a, const lg_logp_args &p, hipStream_t st) {
    const int64_t units = (int64_t)a.M * a.slices;
    if (a.slices > 1) {
        lg_launches(a, units, [&](unsigned n) { logprobs_kernel<T, 0, true><<<n, LG_THREADS, 0, st>>>(a, p); });
        lg_launches(a, units, [&](unsigned n) { logprobs_grad_kernel<T, true, ENTROPY><<<n, LG_THREADS, 0, st>>>(a, p); });
    } else {
        lg_launches(a, units, [&](unsigned n) { logprobs_grad_kernel<T, false, ENTROPY><<<n, LG_THREADS, 0, st>>>(a, p); });
    }
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
