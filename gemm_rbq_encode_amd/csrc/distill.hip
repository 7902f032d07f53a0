// distill.hip -- distillation from a teacher's top log probabilities: the loss
// of rows of logits x [M][V] and its gradient.
#include <hip/hip_runtime.h>

#include "rbq.h"
#include "rbq_kernels.h"
#include "logits_device.h"

namespace rbq {

namespace {

// The teacher names slots (i_j, t_j), j < k.  p_j = e^t_j, with the rest
// r = max(0, 1 - sum p) as one more class (tail), or p_j = e^t_j / sum e^t.
//   L = sum_j p_j (ln p_j - ln q_{i_j}) + r (ln r - ln q_r)
//   q = softmax(x / T),  q_r = the students' mass on the tokens not named
//   dL/dx_v = (1/T) ((P + r) q_v - sum_{j: i_j = v} p_j - [v not named] r q_v / q_r)
// What depends on the slots alone is computed in 64 bits: 1 - sum p cancels.

struct lg_distill_args {
    const int32_t *index;
    const float *t_logp;
    int slots;
    int tail;
    float *loss;
    const float *d_loss;
    void *dx;
    int64_t d_stride;
};

constexpr int LG_MAP = 1 << 15;     // vectors that one map of named tokens covers

struct lg_slots {
    int index[RBQ_TOP_MAX];         // -1: not used
    float x[RBQ_TOP_MAX];           // the student's logit
    double p[RBQ_TOP_MAX];
    double red[LG_WAVES][2];
    int bad, any;
};

__device__ __forceinline__ double lg_block_sum(double v, double (*red)[2], int which) {
    v = wave_sum_f64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6][which] = v;
    __syncthreads();
    double t = 0.0;
    for (int i = 0; i < LG_WAVES; ++i)
        t += red[i][which];
    return t;
}

// The workgroup's sums over a slice; the bits of the named tokens in it are set
// in `map`, a chunk of LG_MAP vectors at a time.
template <typename T, int KIND, bool QUICK>
__device__ __forceinline__ lg_row distill_sums(const typename T::bits *x, const lg_range &r, const lg_slots &sl,
                                               int slots, float c, uint32_t *map, float4 *part) {
    const int tid = threadIdx.x;
    lg_sums<QUICK> s;
    float best;
    int where;
    if constexpr (KIND == LG_NAMED) {
        for (int v0 = r.v0; v0 < r.v1; v0 += LG_MAP) {
            lg_range q = r;
            q.v0 = v0;
            q.v1 = min(r.v1, v0 + LG_MAP);
            for (int i = tid; i < (q.v1 - q.v0 + 3) / 4; i += LG_THREADS)
                map[i] = 0;
            __syncthreads();
            if (tid < slots) {
                const int i = sl.index[tid];
                const int bit = i - q.v0 * LG_VEC;
                if (i >= 0 && bit >= 0 && i / LG_VEC < q.v1)
                    atomicOr(&map[bit >> 5], 1u << (bit & 31));
            }
            __syncthreads();
            lg_walk<T, 0> walk(x, q);
            lg_stream<T, KIND, false>(walk, c, (const uint8_t *)map, q.v0, s, best, where);
            __syncthreads();
        }
    } else {
        lg_walk<T, 0> walk(x, r);
        lg_stream<T, KIND, false>(walk, c, nullptr, 0, s, best, where);
    }
    const lg_sums<QUICK> t = lg_join_block<KIND>(s, c, part);
    if constexpr (QUICK)
        if (!lg_good(t))
            return {t.m, __builtin_nanf(""), 0.0f, true};
    return lg_row_of(t);
}

// dx = e w of a slice.
template <typename T, bool QUICK>
__device__ __forceinline__ void distill_write(const typename T::bits *x, typename T::bits *dx, const lg_range &r,
                                              float m, float c, float w) {
    lg_walk<T, 0> walk(x, r);
    walk.down(dx, [&](float(&e)[LG_VEC], int) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LG_VEC; ++i)
            e[i] = __builtin_amdgcn_exp2f(lg_exponent<QUICK>(e[i], m, c)) * w;
    });
}

// WHOLE: a row per workgroup; SUMS: the sums of a slice; REST: what follows from
// the slices' sums.  GRAD: the gradient of a slice is written (WHOLE, REST).
enum { DS_WHOLE = 0, DS_SUMS = 1, DS_REST = 2 };

template <typename T, int KIND, int MODE, bool GRAD>
__global__ __launch_bounds__(LG_THREADS) void distill_kernel(lg_row_args a, lg_distill_args p) {
    __shared__ float4 part[MODE == DS_REST ? LG_SLICES_MAX : LG_WAVES];
    __shared__ lg_slots sl;
    extern __shared__ uint32_t map[];
    const int tid = threadIdx.x;
    const int per_row = MODE == DS_REST && !GRAD ? 1 : a.slices;
    for (int64_t u = blockIdx.x; u < (int64_t)a.M * per_row; u += gridDim.x) {
        const int row = (int)(u / per_row), slice = (int)(u - (int64_t)row * per_row);
        const typename T::bits *x = (const typename T::bits *)a.x + row * a.stride;
        const lg_range r = lg_slice(a.V, a.slices, slice);
        // the slots
        if (tid == 0)
            sl.bad = sl.any = 0;
        __syncthreads();
        double lp = -__builtin_inf();
        if (tid < p.slots) {
            int i = p.index[(int64_t)row * p.slots + tid];
            const float t = p.t_logp[(int64_t)row * p.slots + tid];
            if (i >= a.V) {
                sl.bad = 1;
                i = -1;
                if (a.status != nullptr)
                    atomicOr(a.status, RBQ_STATUS_BAD_TOKEN);
            } else if (i < 0 || t == -__builtin_inff()) {
                i = -1;
            } else {
                lp = t;
                sl.any = 1;
                // (x may be the gradient's buffer: the slices keep the logits beside their sums)
                float *kept = a.named + (int64_t)row * p.slots + tid;
                if (MODE == DS_WHOLE)
                    sl.x[tid] = T::one(x[i]);
                else if (MODE == DS_REST)
                    sl.x[tid] = *kept;
                else if (i / LG_VEC >= r.v0 && i / LG_VEC < r.v1)
                    *kept = T::one(x[i]);
            }
            sl.index[tid] = i;
        }
        __syncthreads();
        // the row's sums
        lg_row t;
        if constexpr (MODE == DS_REST) {
            for (int i = tid; i < a.slices; i += LG_THREADS)
                part[i] = a.sums[(int64_t)row * a.slices + i];
            __syncthreads();
            t = lg_row_of(lg_join_list<KIND, false>(part, a.slices, a.c));
        } else if constexpr (MODE == DS_SUMS) {
            t = distill_sums<T, KIND, false>(x, r, sl, p.slots, a.c, map, part);
            if (tid == 0)
                a.sums[u] = make_float4(t.m, t.S, t.b, 0.0f);
            __syncthreads();
            continue;
        } else {
            t = distill_sums<T, KIND, true>(x, r, sl, p.slots, a.c, map, part);
            if (t.S != t.S) {
                __syncthreads();
                t = distill_sums<T, KIND, false>(x, r, sl, p.slots, a.c, map, part);
            }
        }
        // the teacher's side
        double top = 0.0;
        if (KIND != LG_NAMED) {     // normalised over the slots: relative to the largest
            const float big = lg_wave_max((float)lp);
            if ((tid & 63) == 0)
                sl.red[tid >> 6][0] = big;
            __syncthreads();
            top = sl.red[0][0];
            for (int i = 1; i < LG_WAVES; ++i)
                top = fmax(top, sl.red[i][0]);
            __syncthreads();
        }
        const bool used = lp != -__builtin_inf();      // (a NaN is used)
        double pj = used ? exp(lp - top) : 0.0;
        double lpj = lp - top;
        double P = lg_block_sum(pj, sl.red, 0), rest = 0.0;
        if (KIND != LG_NAMED) {
            if (sl.any) {
                pj /= P;
                lpj -= log(P);
                P = P != P ? P : 1.0;
            }
        } else {
            rest = 1.0 - P;
            rest = rest > 0.0 ? rest : rest != rest ? rest : 0.0;
        }
        // the student's side, the loss
        const double S = KIND == LG_NAMED ? (double)t.S + (double)t.b : (double)t.S;
        const double logS = log(S), c = (double)a.c;
        double term = 0.0;
        if (used && pj != 0.0) {
            const double xj = sl.x[tid], m = t.m, d = t.quick ? xj * c - m : (xj - m) * c;
            term = pj * (lpj - (S == 0.0 ? -__builtin_inf() : d * 0.6931471805599453 - logS));
        }
        double loss = lg_block_sum(term, sl.red, 1);
        if (KIND == LG_NAMED && rest != 0.0)
            loss = S == 0.0 ? __builtin_inf() : loss + rest * (log(rest) - (log((double)t.S) - logS));
        if (sl.bad)
            loss = __builtin_nan("");
        if (tid == 0 && slice == 0 && p.loss != nullptr)
            p.loss[row] = (float)loss;
        if constexpr (GRAD) {
            typename T::bits *dx = (typename T::bits *)p.dx + row * p.d_stride;
            const float d = p.d_loss[row];
            if (d == 0.0f || S == 0.0 || (KIND != LG_NAMED && !sl.any && !sl.bad)) {
                lg_zero<T>(dx, r);
            } else {
                const double by = sl.bad ? __builtin_nan("") : (double)d * (double)a.inv_t;
                const double all = by * (P + rest) / S;         // per e of a named token
                const double away = KIND == LG_NAMED && rest != 0.0 && t.S != 0.0f ? by * rest / (double)t.S : 0.0;
                if (used)
                    sl.p[tid] = pj;
                __syncthreads();    // every slot's logit has been read: dx may be x
                if (MODE == DS_WHOLE && t.quick)
                    distill_write<T, true>(x, dx, r, t.m, a.c, (float)(all - away));
                else
                    distill_write<T, false>(x, dx, r, t.m, a.c, (float)(all - away));
                __syncthreads();    // then the named tokens, each thread a slot; a token named twice gets both in each
                if (used && sl.index[tid] / LG_VEC >= r.v0 && sl.index[tid] / LG_VEC < r.v1) {
                    const int i = sl.index[tid];
                    double mine = 0.0;
                    for (int j = 0; j < p.slots; ++j)
                        mine += sl.index[j] == i ? sl.p[j] : 0.0;
                    const double e = __builtin_amdgcn_exp2f(t.exponent(sl.x[tid], a.c));
                    dx[i] = T::of((float)(e * all - by * mine));
                }
            }
        }
        __syncthreads();
    }
}

template <typename T, int KIND, bool GRAD>
hipError_t distill_of(lg_row_args a, const lg_distill_args &p, hipStream_t st) {
    const unsigned grid = lg_grid((int64_t)a.M * a.slices), rows = lg_grid(a.M);
    const int vectors = (a.V + LG_VEC - 1) / LG_VEC, each = (vectors + a.slices - 1) / a.slices;
    const size_t map = KIND == LG_NAMED ? (size_t)((each < LG_MAP ? each : LG_MAP) + 3) / 4 * 4 : 0;
    if (a.slices == 1) {
        distill_kernel<T, KIND, DS_WHOLE, GRAD><<<grid, LG_THREADS, map, st>>>(a, p);
    } else {
        distill_kernel<T, KIND, DS_SUMS, false><<<grid, LG_THREADS, map, st>>>(a, p);
        distill_kernel<T, KIND, DS_REST, GRAD><<<GRAD ? grid : rows, LG_THREADS, 0, st>>>(a, p);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t distill_any(const lg_row_args &a, const lg_distill_args &p, hipStream_t st) {
    if (p.tail)
        return p.dx != nullptr ? distill_of<T, LG_NAMED, true>(a, p, st) : distill_of<T, LG_NAMED, false>(a, p, st);
    return p.dx != nullptr ? distill_of<T, LG_PLAIN, true>(a, p, st) : distill_of<T, LG_PLAIN, false>(a, p, st);
}

}  // namespace

hipError_t launch_distill(const void *x, uint32_t type, int M, int V, int64_t stride, float temperature,
                          const int32_t *index, const float *t_logp, int slots, int tail, float *loss,
                          const float *d_loss, void *dx, int64_t d_stride, void *workspace, size_t bytes,
                          int32_t *status, hipStream_t st) {
    lg_row_args a = row_args(x, M, V, stride, temperature, status);
    lg_distill_args p = {};
    p.index = index;
    p.t_logp = t_logp;
    p.slots = slots;
    p.tail = tail;
    p.loss = loss;
    p.d_loss = d_loss;
    p.dx = dx;
    p.d_stride = d_stride;
    cut_rows(a, 0, slots, workspace, bytes);
    return type == RBQ_L_F16   ? distill_any<lg_f16>(a, p, st)
           : type == RBQ_L_F32 ? distill_any<lg_f32>(a, p, st)
                               : distill_any<lg_bf16>(a, p, st);
}

}  // namespace rbq
