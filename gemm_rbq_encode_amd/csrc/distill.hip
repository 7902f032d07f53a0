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

// What the slots of a row say, in LDS.  One wave forms it, two slots a lane,
// while the others read the row.
struct lg_slots {
    int index[RBQ_TOP_MAX];     // -1: not used
    float x[RBQ_TOP_MAX];       // the student's logit
    double p[RBQ_TOP_MAX];      // 0: not used
    double P, rest, own;        // sum of p, the rest, sum of p ln p over the slots
    int bad, any;
};

// The workgroup's sums over a slice; the bits of the named tokens in it are set
// in `map`, a chunk of LG_MAP vectors at a time.
template <typename T, int KIND, bool QUICK, int TH>
__device__ __forceinline__ lg_row distill_sums(const typename T::bits *x, const lg_range &r, const lg_slots &sl,
                                               int slots, float c, uint32_t *map, float4 *part,
                                               void *held) {
    const int tid = threadIdx.x;
    lg_sums<QUICK> s;
    float best;
    int where;
    if constexpr (KIND == LG_NAMED) {
        for (int v0 = r.v0; v0 < r.v1; v0 += LG_MAP) {
            lg_range q = r;
            q.v0 = v0;
            q.v1 = min(r.v1, v0 + LG_MAP);
            for (int i = tid; i < (q.v1 - q.v0 + 3) / 4; i += TH)
                map[i] = 0;
            __syncthreads();
            for (int j = tid; j < slots; j += TH) {
                const int i = sl.index[j];
                const int bit = i - q.v0 * LG_VEC;
                if (i >= 0 && bit >= 0 && i / LG_VEC < q.v1)
                    atomicOr(&map[bit >> 5], 1u << (bit & 31));
            }
            __syncthreads();
            lg_walk<T, TH> walk(x, q, held);
            lg_stream<T, KIND, false>(walk, c, (const uint8_t *)map, q.v0, s, best, where);
            __syncthreads();
        }
    } else {
        lg_walk<T, TH> walk(x, r, held);
        lg_stream<T, KIND, false>(walk, c, nullptr, 0, s, best, where);
    }
    const lg_sums<QUICK> t = lg_join_block<KIND, TH>(s, c, part);
    if constexpr (QUICK)
        if (!lg_good(t))
            return {t.m, __builtin_nanf(""), 0.0f, true};
    return lg_row_of(t);
}

// dx = e w of a slice; FAR: e up w.
template <typename T, bool QUICK, bool FAR, int TH>
__device__ __forceinline__ void distill_write(const typename T::bits *x, typename T::bits *dx, const lg_range &r,
                                              float m, float c, float up, float w, void *held) {
    lg_walk<T, TH> walk(x, r, held);
    walk.down(dx, [&](float(&e)[LG_VEC], int) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LG_VEC; ++i) {
            const float v = __builtin_amdgcn_exp2f(lg_exponent<QUICK>(e[i], m, c));
            e[i] = (FAR ? v * up : v) * w;
        }
    });
}

// A weight beyond fp32 -- the rest's share over a sum S of far entries alone -- goes in two
// factors: up, the power of two that brings S to 1 .. 2, and what is left, which is of
// the size of the gradient.  (A named token's e up may be infinite: it is written after.)
template <typename T, bool QUICK, int TH>
__device__ __forceinline__ void distill_scaled(const typename T::bits *x, typename T::bits *dx, const lg_range &r,
                                               const lg_row &t, float c, double w, void *held) {
    if (__builtin_fabs(w) < 0x1p127) {
        distill_write<T, QUICK, false, TH>(x, dx, r, t.m, c, 1.0f, (float)w, held);
    } else {
        const int k = max(0, 127 - (int)(__builtin_bit_cast(uint32_t, t.S) >> 23));     // (S is normal)
        distill_write<T, QUICK, true, TH>(x, dx, r, t.m, c, ldexpf(1.0f, k), (float)ldexp(w, -k), held);
    }
}

// WHOLE: a row per workgroup; SUMS: the sums of a slice; REST: what follows from
// the slices' sums.  GRAD: the gradient of a slice is written (WHOLE, REST).
enum { DS_WHOLE = 0, DS_SUMS = 1, DS_REST = 2 };

// The slots' tokens.
__device__ __forceinline__ void distill_slots(int row, const lg_row_args &a, const lg_distill_args &p, float (&t)[2],
                                              lg_slots &sl) {
    const int lane = threadIdx.x & 63;
    const int64_t first = (int64_t)row * p.slots;
    int index[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = lane + 64 * q;
        index[q] = j < p.slots ? p.index[first + j] : -1;
        t[q] = j < p.slots ? p.t_logp[first + j] : -__builtin_inff();
    }
    bool bad = false, any = false, beyond = false;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = lane + 64 * q;
        beyond |= index[q] >= a.V;
        bad |= index[q] >= a.V && t[q] != -__builtin_inff();    // (else not used)
        if (index[q] < 0 || index[q] >= a.V || t[q] == -__builtin_inff()) {
            index[q] = -1;
            t[q] = -__builtin_inff();
        }
        any |= index[q] >= 0;
        sl.index[j] = index[q];
    }
    bad = __any(bad);
    any = __any(any);
    beyond = __any(beyond);
    if (lane == 0) {
        sl.bad = bad;
        sl.any = any;
        if (beyond && a.status != nullptr)
            atomicOr(a.status, RBQ_STATUS_BAD_TOKEN);
    }
}

// The student's logits of the slots' tokens: x may be the gradient's buffer, so the
// slices keep them beside their sums.  A wave's part, behind the barrier that the
// others wait at for the tokens alone.
template <typename T, int MODE>
__device__ __forceinline__ void distill_logits(const typename T::bits *x, const lg_range &r, int row,
                                               const lg_row_args &a, const lg_distill_args &p, lg_slots &sl) {
    const int lane = threadIdx.x & 63;
    const int64_t first = (int64_t)row * p.slots;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = lane + 64 * q, i = sl.index[j];
        if (i < 0)
            continue;
        if (MODE == DS_WHOLE)
            sl.x[j] = T::one(x[i]);
        else if (MODE == DS_REST)
            sl.x[j] = a.named[first + j];
        else if (i / LG_VEC >= r.v0 && i / LG_VEC < r.v1)
            a.named[first + j] = T::one(x[i]);
    }
}

// The teacher's side, from the slots' log probabilities t (-inf: not used).
template <int KIND>
__device__ __forceinline__ void distill_teacher(const float (&t)[2], int slots, lg_slots &sl) {
    const int lane = threadIdx.x & 63;
    // normalised over the slots: relative to the largest
    const double top = KIND == LG_NAMED ? 0.0 : (double)lg_wave_max(fmaxf(t[0], t[1]));
    double lp[2], pj[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        lp[q] = (double)t[q] - top;
        pj[q] = t[q] == -__builtin_inff() ? 0.0 : exp(lp[q]);   // (a NaN counts)
    }
    double P = wave_sum_f64_dpp(pj[0] + pj[1]), rest = 0.0;
    if (KIND != LG_NAMED) {
        if (P != 0.0) {
            const double by = 1.0 / P, less = log(P);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                pj[q] *= by;
                lp[q] -= less;
            }
            P = P != P ? P : 1.0;
        }
    } else {
        rest = 1.0 - P;
        rest = rest > 0.0 ? rest : rest != rest ? rest : 0.0;
    }
    double own = wave_sum_f64_dpp((pj[0] != 0.0 ? pj[0] * lp[0] : 0.0) + (pj[1] != 0.0 ? pj[1] * lp[1] : 0.0));
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (lane + 64 * q < slots)
            sl.p[lane + 64 * q] = pj[q];
    if (lane == 0) {
        sl.P = P;
        sl.rest = rest;
        sl.own = own;
    }
}

// The teacher's rest: what rounding of its log probabilities can leave (their sum is
// off by up to 2^-15) is none where the student has no mass on the tokens not named --
// all tokens are named, or both mask the others.
template <int KIND>
__device__ __forceinline__ double distill_rest(const lg_row &t, const lg_slots &sl) {
    return KIND != LG_NAMED || (t.S == 0.0f && sl.rest <= 0x1p-15) ? 0.0 : sl.rest;
}

// A wave's part: the loss of the row, sum p ln p - sum p ln q.
template <int KIND>
__device__ __forceinline__ float distill_loss(const lg_row &t, double S, float cf, int slots, const lg_slots &sl) {
    const int lane = threadIdx.x & 63;
    const double c = cf, m = t.m;
    double cross = 0.0;             // sum p ln e
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = lane + 64 * q;
        const double pj = j < slots ? sl.p[j] : 0.0;
        if (pj != 0.0) {
            const double x = sl.x[j];
            cross += pj * ((t.quick ? x * c - m : (x - m) * c) * 0.6931471805599453);
        }
    }
    cross = wave_sum_f64_dpp(cross);
    if (sl.bad)
        return __builtin_nanf("");
    const double rest = distill_rest<KIND>(t, sl);
    if (sl.P == 0.0 && rest == 0.0)
        return 0.0f;
    if (S == 0.0)
        return sl.P + rest != sl.P + rest ? __builtin_nanf("") : __builtin_inff();
    const double logS = log(S);
    double loss = sl.own - cross + sl.P * logS;
    if (KIND == LG_NAMED && rest != 0.0)
        loss += rest * (log(rest) - (log((double)t.S) - logS));
    return (float)loss;
}

// A row a workgroup (or a slice, and the rest in a second launch); the teacher's side
// by wave 0 while the others read logits.  The named tokens are marked in a map of bits
// in LDS, and their exponentials left out of the sum of the rest as it is formed: 1 -
// sum q would cancel.  Bound by the read and the write of the gradient: a step of 2048 x
// 128256 fp16 with 64 slots and the tail 240 to 247 us (4.3 TB/s of both, a copy 5.2),
// the loss alone 98 (5.4 TB/s); 64 x 128256 fp32 13.5, of it 9.1 the slices' sums and
// 4.4 the second launch; 77 x 32001 bf16 12 on the device.
template <typename T, int KIND, int MODE, bool GRAD, int TH>
__global__ __launch_bounds__(TH) void distill_kernel(lg_row_args a, lg_distill_args p) {
    __shared__ float4 part[MODE == DS_REST ? LG_SLICES_MAX : TH / 64];
    __shared__ lg_slots sl;
    __shared__ uint4 held_[GRAD && MODE == DS_WHOLE ? lg_walk<T, TH>::HELD_BYTES / 16 : 1];
    extern __shared__ uint32_t map[];
    const int tid = threadIdx.x;
    const int per_row = MODE == DS_REST && !GRAD ? 1 : a.slices;
    const int64_t u = a.first + blockIdx.x;
    const int row = (int)(u / per_row), slice = (int)(u - (int64_t)row * per_row);
    const typename T::bits *x = (const typename T::bits *)a.x + row * a.stride;
    const lg_range r = lg_slice(a.V, a.slices, slice);
    // (a row in several maps is not held: its walks up end elsewhere)
    uint4 *const held = GRAD && MODE == DS_WHOLE && (KIND != LG_NAMED || r.v1 <= LG_MAP) ? held_ : nullptr;
    float t_logp[2];
    if (tid < 64)
        distill_slots(row, a, p, t_logp, sl);
    __syncthreads();
    if (tid < 64) {
        distill_logits<T, MODE>(x, r, row, a, p, sl);
        if (MODE != DS_SUMS)
            distill_teacher<KIND>(t_logp, p.slots, sl);
    }
    lg_row t;
    if constexpr (MODE == DS_REST) {
        for (int i = tid; i < a.slices; i += TH)
            part[i] = a.sums[(int64_t)row * a.slices + i];
        __syncthreads();
        t = lg_row_of(lg_join_list<KIND, false>(part, a.slices, a.c));
    } else if constexpr (MODE == DS_SUMS) {
        t = distill_sums<T, KIND, false, TH>(x, r, sl, p.slots, a.c, map, part, held);
        if (tid == 0)
            a.sums[u] = make_float4(t.m, t.S, t.b, 0.0f);
        return;
    } else {
        t = distill_sums<T, KIND, true, TH>(x, r, sl, p.slots, a.c, map, part, held);
        if (t.S != t.S) {
            __syncthreads();
            t = distill_sums<T, KIND, false, TH>(x, r, sl, p.slots, a.c, map, part, held);
        }
    }
    // (what is left of entries farther than fp32's exponents go is none: their e is 0 below)
    if (KIND == LG_NAMED && t.S < 0x1p-126f)
        t.S = 0.0f;
    const double S = KIND == LG_NAMED ? (double)t.S + (double)t.b : (double)t.S;
    if (tid < 64 && slice == 0 && p.loss != nullptr) {
        const float loss = distill_loss<KIND>(t, S, a.c, p.slots, sl);
        if (tid == 0)
            p.loss[row] = loss;
    }
    if constexpr (GRAD) {
        typename T::bits *dx = (typename T::bits *)p.dx + row * p.d_stride;
        const float d = p.d_loss[row];
        if (d == 0.0f || (!sl.bad && (S == 0.0 || (KIND != LG_NAMED && !sl.any)))) {
            lg_zero<T, TH>(dx, r);
            return;
        }
        const double by = sl.bad ? __builtin_nan("") : (double)d * (double)a.inv_t;
        const double rest = distill_rest<KIND>(t, sl);
        const double all = by * (sl.P + rest) / S;          // per e of a named token
        const double away = KIND == LG_NAMED && rest != 0.0 && t.S != 0.0f ? by * rest / (double)t.S : 0.0;
        // (every slot's logit has been read: dx may be x)
        if (MODE == DS_WHOLE && t.quick)
            distill_scaled<T, true, TH>(x, dx, r, t, a.c, all - away, held);
        else
            distill_scaled<T, false, TH>(x, dx, r, t, a.c, all - away, held);
        __syncthreads();    // then the named tokens, a thread a slot; a token named twice gets both in each
        for (int j = tid; j < p.slots; j += TH) {
            const int i = sl.index[j];
            if (i < 0 || i / LG_VEC < r.v0 || i / LG_VEC >= r.v1)
                continue;
            double mine = 0.0;
            for (int k = 0; k < p.slots; k += 8) {      // (8 reads on their way at a time; slots behind the last: -1)
                int same[8];
                double pk[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    same[q] = sl.index[k + q];
                    pk[q] = sl.p[k + q];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    mine += same[q] == i ? pk[q] : 0.0;
            }
            const double e = __builtin_amdgcn_exp2f(t.exponent(sl.x[j], a.c));
            dx[i] = T::of((float)(e * all - by * mine));
        }
    }
}

template <typename T, int KIND, bool GRAD>
hipError_t distill_of(lg_row_args a, const lg_distill_args &p, hipStream_t st) {
    const int64_t units = (int64_t)a.M * a.slices;
    const int vectors = (a.V + LG_VEC - 1) / LG_VEC, each = (vectors + a.slices - 1) / a.slices;
    const size_t map = KIND == LG_NAMED ? (size_t)((each < LG_MAP ? each : LG_MAP) + 3) / 4 * 4 : 0;
    auto run = [&](auto th) {
        constexpr int TH = decltype(th)::value;
        if (a.slices == 1) {
            lg_launches(a, units, [&](unsigned n) {
                distill_kernel<T, KIND, DS_WHOLE, GRAD, TH><<<n, TH, map, st>>>(a, p);
            });
        } else {
            lg_launches(a, units, [&](unsigned n) {
                distill_kernel<T, KIND, DS_SUMS, false, TH><<<n, TH, map, st>>>(a, p);
            });
            lg_launches(a, GRAD ? units : a.M, [&](unsigned n) {
                distill_kernel<T, KIND, DS_REST, GRAD, TH><<<n, TH, 0, st>>>(a, p);
            });
        }
    };
    const int threads = logits_threads(each, 0);
    if (threads == 512)
        run(std::integral_constant<int, 512>{});
    else if (threads == 256)
        run(std::integral_constant<int, 256>{});
    else
        run(std::integral_constant<int, 128>{});
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
