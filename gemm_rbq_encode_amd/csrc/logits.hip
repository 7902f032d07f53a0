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

// The largest k entries of a slice, sorted, in lists[0 .. 64 E) (LDS; ends with
// a barrier), for every row whatever its values at a bounded cost: each thread
// knows its largest entry, and the k largest entries lie with the k threads
// whose largest entries are largest (any other has k better ones before it).
// Those threads' vectors are read once more, from the caches, by all threads,
// and what is below the k-th of those maxima is dropped.
template <typename T, int E>
__device__ __forceinline__ void lg_select(const typename T::bits *x, const lg_range &r, int k, float best, int where,
                                          uint64_t *lists, uint64_t *waiting) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t n[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        n[e] = 0;
    n[0] = lg_key(best, where * LG_VEC + LG_VEC - 1);
    lg_sort<E>(n);
    lg_block_merge<E, LG_WAVES>(n, lists);
    uint64_t least = lists[k - 1];
    least = least == 0 ? 1 : least;
    int groups = 0;     // threads to look at: those with an entry at all
#pragma unroll
    for (int e = 0; e < E; ++e)
        groups += __popcll(__ballot(e * 64 + lane < k && lists[e * 64 + lane] != 0));
    const int turns = (r.v1 - r.v0 + LG_THREADS - 1) / LG_THREADS;
    lg_top<E> top;
    top.start(waiting + wave * 64 * E);
    for (int q0 = wave * 64; q0 < groups * turns; q0 += LG_THREADS) {
        const int q = q0 + lane;
        float e[LG_VEC];
        int v = r.v1;
        if (q < groups * turns) {
            const int g = q / turns;
            v = r.v0 + (((lg_index(lists[g]) / LG_VEC) - r.v0) & (LG_THREADS - 1)) + (q - g * turns) * LG_THREADS;
        }
        if (v >= r.v1) {
#pragma unroll
            for (int i = 0; i < LG_VEC; ++i)
                e[i] = -__builtin_inff();
        } else if (v < r.whole) {
            lg_values<T>(lg_load<T>(x + (int64_t)v * LG_VEC), e);
        } else {
            lg_load_part<T>(x + (int64_t)v * LG_VEC, r.rest, e);
        }
#pragma unroll
        for (int i = 0; i < LG_VEC; ++i) {
            const uint64_t key = lg_key(e[i], v * LG_VEC + i);
            top.offer(key, key >= least);
        }
    }
    top.settle();
    __syncthreads();    // the lists have been read
    lg_block_merge<E, LG_WAVES>(top.k, lists);
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
template <typename T, bool TOP, int KEEP>
__device__ __forceinline__ lg_row lg_whole_row(lg_walk<T, KEEP> &walk, float c, float4 *part, float &best, int &where) {
    {
        lg_sums<true> s;
        lg_stream<T, LG_ENTROPY, TOP>(walk, c, nullptr, 0, s, best, where);
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
    constexpr int N = LG_WAVES * 64 * (E > 0 ? E : 1);
    __shared__ float4 part[LG_WAVES];
    __shared__ uint64_t lists[E > 0 ? N : 1], waiting[E > 0 ? N : 1];
    for (int64_t u = blockIdx.x; u < (int64_t)a.M * a.slices; u += gridDim.x) {
        const int row = (int)(u / a.slices), slice = (int)(u - (int64_t)row * a.slices);
        const typename T::bits *x = (const typename T::bits *)a.x + row * a.stride;
        const lg_range r = lg_slice(a.V, a.slices, slice);
        const int64_t target = p.targets == nullptr ? -1 : p.targets[row];
        float best = -__builtin_inff();
        int where = 0;
        lg_walk<T, 0> walk(x, r);
        lg_row sums;
        if constexpr (SLICED) {
            lg_sums<false> s;
            lg_stream<T, LG_ENTROPY, (E > 0)>(walk, a.c, nullptr, 0, s, best, where);
            sums = lg_row_of(lg_join_block<LG_ENTROPY>(s, a.c, part));
        } else {
            sums = lg_whole_row<T, (E > 0)>(walk, a.c, part, best, where);
        }
        if constexpr (E > 0)
            lg_select<T, E>(x, r, p.top, best, where, lists, waiting);
        if constexpr (SLICED) {
            if (threadIdx.x == 0) {
                const bool here = lg_inside(target, a.V) && target >= (int64_t)r.v0 * LG_VEC &&
                                  target < (int64_t)r.v1 * LG_VEC;
                a.sums[u] = make_float4(sums.m, sums.S, sums.b, here ? T::one(x[target]) : 0.0f);
            }
            if constexpr (E > 0)
                for (int j = threadIdx.x; j < p.top; j += LG_THREADS)
                    a.keys[u * p.top + j] = lists[j];
        } else {
            const lg_logp_row w(sums);
            if (threadIdx.x == 0)
                lg_write_logp(w, lg_inside(target, a.V) ? T::one(x[target]) : 0.0f, target, row, a, p);
            if constexpr (E > 0)
                lg_write_top(w, lists, row, a.c, a.inv_t, p);
        }
        __syncthreads();    // before the next unit writes LDS
    }
}

// The slices of a row joined.
template <int E>
__global__ __launch_bounds__(LG_THREADS) void logprobs_join_kernel(lg_row_args a, lg_logp_args p) {
    constexpr int N = LG_WAVES * 64 * (E > 0 ? E : 1);
    __shared__ float4 part[LG_SLICES_MAX];
    __shared__ uint64_t lists[E > 0 ? N : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int row = blockIdx.x; row < a.M; row += gridDim.x) {
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
        __syncthreads();
    }
}

// The gradient of sum_m a_m logp_m + b_m H_m:
//   dx_v = (a ([v = target] - p_v) - b p_v (ln p_v + H)) / T
// with p_v = e_v / S and ln p_v = ln 2 (d_v - log2 S), so that the part without
// the target is e_v (w0 + w1 d_v).  Where rows are whole the sums are formed here,
// and the second pass over the row finds it in the caches.
template <typename T, bool QUICK, bool ENTROPY, int KEEP>
__device__ __forceinline__ void lg_logp_grad(lg_walk<T, KEEP> &walk, typename T::bits *dx, float m, float c, float w0,
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

template <typename T, int KEEP, bool SLICED, bool ENTROPY>
__global__ __launch_bounds__(LG_THREADS) void logprobs_grad_kernel(lg_row_args a, lg_logp_args p) {
    __shared__ float4 part[LG_SLICES_MAX];
    for (int64_t u = blockIdx.x; u < (int64_t)a.M * a.slices; u += gridDim.x) {
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
            continue;
        }
        lg_walk<T, KEEP> walk(x, r);
        lg_row sums;
        if constexpr (SLICED) {
            for (int i = threadIdx.x; i < a.slices; i += LG_THREADS)
                part[i] = a.sums[(int64_t)row * a.slices + i];
            __syncthreads();
            sums = lg_row_of(lg_join_list<LG_ENTROPY, false>(part, a.slices, a.c));
        } else {
            float best;
            int where;
            sums = lg_whole_row<T, false>(walk, a.c, part, best, where);
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
}

template <typename T>
hipError_t logprobs_of(lg_row_args a, const lg_logp_args &p, hipStream_t st) {
    const unsigned grid = lg_grid((int64_t)a.M * a.slices), rows = lg_grid(a.M);
    auto run = [&](auto e) {
        constexpr int E = decltype(e)::value;
        if (a.slices > 1) {
            logprobs_kernel<T, E, true><<<grid, LG_THREADS, 0, st>>>(a, p);
            logprobs_join_kernel<E><<<rows, LG_THREADS, 0, st>>>(a, p);
        } else {
            logprobs_kernel<T, E, false><<<grid, LG_THREADS, 0, st>>>(a, p);
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

template <typename T>
hipError_t logprobs_grad_of(lg_row_args a, const lg_logp_args &p, hipStream_t st) {
    const unsigned grid = lg_grid((int64_t)a.M * a.slices);
    const bool entropy = p.d_entropy != nullptr;
    if (a.slices > 1) {
        logprobs_kernel<T, 0, true><<<grid, LG_THREADS, 0, st>>>(a, p);
        if (entropy)
            logprobs_grad_kernel<T, 0, true, true><<<grid, LG_THREADS, 0, st>>>(a, p);
        else
            logprobs_grad_kernel<T, 0, true, false><<<grid, LG_THREADS, 0, st>>>(a, p);
    } else if (entropy) {
        logprobs_grad_kernel<T, LG_KEEP, false, true><<<grid, LG_THREADS, 0, st>>>(a, p);
    } else {
        logprobs_grad_kernel<T, LG_KEEP, false, false><<<grid, LG_THREADS, 0, st>>>(a, p);
    }
    return hipGetLastError();
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
    return type == RBQ_L_F16   ? logprobs_grad_of<lg_f16>(a, p, st)
           : type == RBQ_L_F32 ? logprobs_grad_of<lg_f32>(a, p, st)
                               : logprobs_grad_of<lg_bf16>(a, p, st);
}

}  // namespace rbq
