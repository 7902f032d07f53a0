// logits_device.h -- device code shared by the kernels that stream rows of
// logits: loads, the running softmax sums of a thread and their joining, and
// the selection of the largest entries.
#pragma once

#include "rbq_device.h"
#include "logits_plan.h"

namespace rbq {

constexpr float LG_LOWEST = -3.402823466e38f;   // the lowest finite float
constexpr float LG_FAR = -1.0e4f;               // exponents below this are 0 in any case

// ---- loads and stores ---------------------------------------------------------
//
// A row starts wherever the stride puts it, so vectors are only aligned like one
// entry; the memory system takes 16-byte accesses at any such address.

typedef uint32_t lg_u32x4 __attribute__((ext_vector_type(4), aligned(2)));

struct lg_f16 {
    static constexpr int SPARE = 13;     // low bits that are equal in all of its values as fp32
    typedef uint16_t bits;
    struct raw {
        lg_u32x4 a;
    };
    static __device__ __forceinline__ float one(uint16_t v) { return h2f(v); }
    static __device__ __forceinline__ uint16_t of(float v) { return f2h(v); }
};
struct lg_bf16 {
    static constexpr int SPARE = 16;     // low bits that are equal in all of its values as fp32
    typedef uint16_t bits;
    struct raw {
        lg_u32x4 a;
    };
    static __device__ __forceinline__ float one(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t of(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct lg_f32 {
    static constexpr int SPARE = 0;     // low bits that are equal in all of its values as fp32
    typedef uint32_t bits;
    struct raw {
        lg_u32x4 a, b;
    };
    static __device__ __forceinline__ float one(uint32_t v) { return __builtin_bit_cast(float, v); }
    static __device__ __forceinline__ uint32_t of(float v) { return __builtin_bit_cast(uint32_t, v); }
};

template <typename T>
__device__ __forceinline__ typename T::raw lg_load(const typename T::bits *p) {
    typename T::raw r;
    r.a = *(const lg_u32x4 *)p;
    if constexpr (sizeof(typename T::bits) == 4)
        r.b = *(const lg_u32x4 *)(p + 4);
    return r;
}

// ... past the caches
template <typename T>
__device__ __forceinline__ typename T::raw lg_load_past(const typename T::bits *p) {
    typename T::raw r;
    r.a = __builtin_nontemporal_load((const lg_u32x4 *)p);
    if constexpr (sizeof(typename T::bits) == 4)
        r.b = __builtin_nontemporal_load((const lg_u32x4 *)(p + 4));
    return r;
}

template <typename T>
__device__ __forceinline__ void lg_values(const typename T::raw &r, float (&x)[LG_VEC]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(typename T::bits) == 4) {
            x[i] = T::one(r.a[i]);
            x[4 + i] = T::one(r.b[i]);
        } else {
            x[2 * i] = T::one((uint16_t)r.a[i]);
            x[2 * i + 1] = T::one((uint16_t)(r.a[i] >> 16));
        }
    }
}

template <typename T>
__device__ __forceinline__ void lg_store(typename T::bits *p, const float (&x)[LG_VEC]) {
    lg_u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(typename T::bits) == 4) {
            a[i] = T::of(x[i]);
            b[i] = T::of(x[4 + i]);
        } else {
            a[i] = (uint32_t)T::of(x[2 * i]) | (uint32_t)T::of(x[2 * i + 1]) << 16;
        }
    }
    __builtin_nontemporal_store(a, (lg_u32x4 *)p);
    if constexpr (sizeof(typename T::bits) == 4)
        __builtin_nontemporal_store(b, (lg_u32x4 *)(p + 4));
}

// The first n < LG_VEC entries at p, -inf behind them.
template <typename T>
__device__ __forceinline__ void lg_load_part(const typename T::bits *p, int n, float (&x)[LG_VEC]) {
#pragma unroll
    for (int i = 0; i < LG_VEC; ++i)
        x[i] = i < n ? T::one(p[i]) : -__builtin_inff();
}

template <typename T>
__device__ __forceinline__ void lg_store_part(typename T::bits *p, int n, const float (&x)[LG_VEC]) {
#pragma unroll
    for (int i = 0; i < LG_VEC; ++i)
        if (i < n)
            p[i] = T::of(x[i]);
}

// Maximum over a wave by DPP: inside quads, mirrored halves and rows of 16, then
// lane 15 of a row to the next one and lane 31 to the upper half; lane 63 has the
// whole.

#define LG_DPP(old, v, ctrl, rows) \
    __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v), ctrl, rows, 0xF, false))

__device__ __forceinline__ float lg_lane63(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ float lg_wave_max(float v) {
    v = fmaxf(v, LG_DPP(v, v, 0xB1, 0xF));
    v = fmaxf(v, LG_DPP(v, v, 0x4E, 0xF));
    v = fmaxf(v, LG_DPP(v, v, 0x141, 0xF));
    v = fmaxf(v, LG_DPP(v, v, 0x140, 0xF));
    v = fmaxf(v, LG_DPP(v, v, RBQ_DPP_ROW_BCAST15, 0xA));
    v = fmaxf(v, LG_DPP(v, v, RBQ_DPP_ROW_BCAST31, 0xC));
    return lg_lane63(v);
}

// ---- running sums ---------------------------------------------------------------
//
// e(x) = 2^d relative to a reference that follows the maximum lazily: it moves
// when an entry lies more than LG_SLACK above it (in the exponent), so e stays
// small and nothing overflows.  With c = log2(e) / T there are two ways to d:
//  * QUICK   d = x c - r, one fma, r = the product top c as it was rounded (what
//            that loses is the same for all entries, and cancels in e / S).  It
//            starts at -LG_FLOOR and is good for rows whose reference ends within
//            -LG_FLOOR / 2 .. LG_FLOOR (there the rounding of r is at most 4) and
//            whose sum is a positive number: lg_good.
//  * otherwise  d = (x - m) c: the difference first, so that rows of the type's
//            lowest value have finite exponents where products with c would be
//            infinite.  Rows that are not good are done once more this way.

constexpr float LG_SLACK = 4.0f;
constexpr float LG_FLOOR = 67108864.0f;     // 2^26

// Kinds of the two sums: of e and of e d; of e alone; of e over the entries
// whose bit of a map is clear and over those whose bit is set.
enum { LG_ENTROPY = 0, LG_PLAIN = 1, LG_NAMED = 2 };

template <bool QUICK>
struct lg_sums {
    float m = QUICK ? -LG_FLOOR : LG_LOWEST, a = 0.0f, b = 0.0f;
};

template <bool QUICK>
__device__ __forceinline__ float lg_exponent(float x, float m, float c) {
    return QUICK ? __builtin_fmaf(x, c, -m) : (x - m) * c;
}

__device__ __forceinline__ bool lg_good(const lg_sums<true> &s) {
    const float all = s.a + __builtin_fabsf(s.b);      // (the second sum is no less than -1 of the first's logarithm)
    return s.m > -0.5f * LG_FLOOR && s.m < LG_FLOOR && all > 0.0f && all < __builtin_inff();
}

template <int KIND, bool QUICK>
__device__ __forceinline__ void lg_move(lg_sums<QUICK> &s, float m, float c) {
    const float d = fmaxf(QUICK ? s.m - m : (s.m - m) * c, LG_FAR);
    const float f = __builtin_amdgcn_exp2f(d);
    if constexpr (KIND == LG_ENTROPY)
        s.b = f * __builtin_fmaf(s.a, d, s.b);
    else
        s.b *= f;
    s.a *= f;
    s.m = m;
}

// `slack`: LG_SLACK in the reference's unit.
template <int KIND, bool QUICK>
__device__ __forceinline__ float lg_add(lg_sums<QUICK> &s, const float (&x)[LG_VEC], float c, float slack,
                                        uint32_t named) {
    const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    const float at = QUICK ? top * c : top;
    if (__any(at > s.m + slack)) {
        if (at > s.m + slack)
            lg_move<KIND>(s, at, c);
    }
    if constexpr (KIND == LG_NAMED) {
        if (__any(named != 0)) {
#pragma unroll
            for (int i = 0; i < LG_VEC; ++i) {
                const float e = __builtin_amdgcn_exp2f(lg_exponent<QUICK>(x[i], s.m, c));
                const bool in = named >> i & 1;
                s.a += in ? 0.0f : e;
                s.b += in ? e : 0.0f;
            }
            return top;
        }
    }
#pragma unroll
    for (int i = 0; i < LG_VEC; ++i) {
        const float d = lg_exponent<QUICK>(x[i], s.m, c);
        const float e = __builtin_amdgcn_exp2f(d);
        s.a += e;
        if constexpr (KIND == LG_ENTROPY)
            s.b = __builtin_fmaf(e, fmaxf(d, LG_FAR), s.b);   // a masked entry's 0 * -inf is 0
    }
    return top;
}

// All lanes' sums (in every lane).  An infinite entry makes m infinite and a
// NaN; fmaxf passes NaN by, the sums keep it.
template <int KIND, bool QUICK>
__device__ __forceinline__ lg_sums<QUICK> lg_join_wave(lg_sums<QUICK> s, float c) {
    lg_move<KIND>(s, lg_wave_max(s.m), c);
    s.a = wave_sum_f32_dpp(s.a);
    if constexpr (KIND != LG_PLAIN)
        s.b = wave_sum_f32_dpp(s.b);
    return s;
}

// n sums joined, by every wave for itself.
template <int KIND, bool QUICK>
__device__ __forceinline__ lg_sums<QUICK> lg_join_list(const float4 *v, int n, float c) {
    lg_sums<QUICK> t;
    for (int i = threadIdx.x & 63; i < n; i += 64) {
        lg_sums<QUICK> s;
        s.m = v[i].x, s.a = v[i].y, s.b = v[i].z;
        const float m = fmaxf(s.m, t.m);
        lg_move<KIND>(s, m, c);
        lg_move<KIND>(t, m, c);
        t.a += s.a;
        t.b += s.b;
    }
    return lg_join_wave<KIND>(t, c);
}

// All threads' sums (in every thread); `part` holds one float4 per wave.
template <int KIND, int TH, bool QUICK>
__device__ __forceinline__ lg_sums<QUICK> lg_join_block(const lg_sums<QUICK> &s, float c, float4 *part) {
    const lg_sums<QUICK> w = lg_join_wave<KIND>(s, c);
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = make_float4(w.m, w.a, w.b, 0.0f);
    __syncthreads();
    return lg_join_list<KIND, QUICK>(part, TH / 64, c);
}

// ---- the largest entries ----------------------------------------------------------
//
// A key orders by value, then by lowest index: the value's bits made monotone
// above the complement of the index.  0 is no entry.

__device__ __forceinline__ uint32_t lg_ordered(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);     // -0 is 0
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float lg_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t lg_key(float v, int index) {
    return v > -__builtin_inff() ? (uint64_t)lg_ordered(v) << 32 | (uint32_t)~index : 0;
}
__device__ __forceinline__ int lg_index(uint64_t key) { return (int)~(uint32_t)key; }

__device__ __forceinline__ uint64_t lg_shfl_xor(uint64_t v, int o) {
    return (uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o) << 32 | (uint32_t)__shfl_xor((int)(uint32_t)v, o);
}

// Lists of 64 E keys, entry e * 64 + lane in k[e], sorted downwards (bitonic).
template <int E>
__device__ __forceinline__ void lg_stage(uint64_t (&k)[E], int size, int stride) {
    const int lane = threadIdx.x & 63;
    if (stride >= 64) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int f = e | stride >> 6;
            if (f != e && f < E) {
                const bool down = ((e * 64 + lane) & size) == 0;
                const uint64_t a = k[e], b = k[f];
                k[e] = (a > b) == down ? a : b;
                k[f] = (a > b) == down ? b : a;
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint64_t other = lg_shfl_xor(k[e], stride);
        const bool larger = ((lane & stride) == 0) == (((e * 64 + lane) & size) == 0);
        k[e] = (other > k[e]) == larger ? other : k[e];
    }
}

template <int E>
__device__ __forceinline__ void lg_sort(uint64_t (&k)[E]) {
#pragma unroll
    for (int size = 2; size <= 64 * E; size *= 2)
#pragma unroll
        for (int stride = size / 2; stride > 0; stride /= 2)
            lg_stage<E>(k, size, stride);
}

// The largest 64 E of two sorted lists, `other` in memory.
template <int E>
__device__ __forceinline__ void lg_merge(uint64_t (&k)[E], const uint64_t *other) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint64_t o = other[64 * E - 1 - (e * 64 + lane)];
        k[e] = o > k[e] ? o : k[e];
    }
#pragma unroll
    for (int stride = 32 * E; stride > 0; stride /= 2)
        lg_stage<E>(k, 128 * E, stride);
}

// Orders the LDS accesses of one wave's lanes.
__device__ __forceinline__ void lg_wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One list per wave -> the workgroup's in lists[0 .. 64 E).  `lists` is LDS of
// WAVES * 64 E keys; ends with a barrier.
template <int E, int WAVES>
__device__ __forceinline__ void lg_block_merge(uint64_t (&k)[E], uint64_t *lists) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t *mine = lists + wave * 64 * E;
#pragma unroll
    for (int n = WAVES; n > 0; n /= 2) {
        if (wave < n) {
            if (n < WAVES)
                lg_merge<E>(k, lists + (wave + n) * 64 * E);
#pragma unroll
            for (int e = 0; e < E; ++e)
                mine[e * 64 + lane] = k[e];
        }
        __syncthreads();
    }
}

// A wave's list of the largest keys offered so far, with those not yet merged
// in waiting: 64 E places of LDS.
template <int E>
struct lg_top {
    uint64_t k[E];
    uint64_t *waiting;
    int count;      // waiting keys
    __device__ __forceinline__ void start(uint64_t *place) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            k[e] = 0;
        waiting = place;
        count = 0;
    }
    __device__ __forceinline__ void settle() {
        if (count == 0)
            return;
        const int lane = threadIdx.x & 63;
        uint64_t n[E];
        lg_wave_sync();
#pragma unroll
        for (int e = 0; e < E; ++e)
            n[e] = e * 64 + lane < count ? waiting[e * 64 + lane] : 0;
        lg_sort<E>(n);
        lg_wave_sync();
#pragma unroll
        for (int e = 0; e < E; ++e)
            waiting[e * 64 + lane] = n[e];
        lg_wave_sync();
        lg_merge<E>(k, waiting);
        lg_wave_sync();
        count = 0;
    }
    // Every lane of the wave calls this; lanes with `has` offer a key.
    __device__ __forceinline__ void offer(uint64_t key, bool has) {
        const uint64_t who = __ballot(has);
        if (who == 0)
            return;
        const int n = __popcll(who);
        if (count + n > 64 * E)
            settle();
        if (has)
            waiting[count + __popcll(who & ((1ull << (threadIdx.x & 63)) - 1))] = key;
        count += n;
    }
};

// ---- rows and slices ----------------------------------------------------------

struct lg_row_args {
    const void *x;
    int64_t first;      // the launch's first row or slice
    int64_t stride;
    int M, V, slices;
    float c, inv_t;     // log2(e) / T, 1 / T
    int32_t *status;
    float4 *sums;       // partial sums [M][slices], the target's logit in the last place
    uint64_t *keys;     // partial lists [M][slices][top]
    float *named;       // logits of the named tokens [M][slots]
};

// The slice of a row that a workgroup works on, in vectors of LG_VEC entries:
// [v0, v1); of those, the row's last one may be part empty.
struct lg_range {
    int v0, v1, whole, rest;    // `whole`: vectors of the row that are full; rest: entries behind them
};

// Vectors of a slice (the last ones may have fewer).
__host__ __device__ __forceinline__ int lg_each(int V, int slices) {
    return ((V + LG_VEC - 1) / LG_VEC + slices - 1) / slices;
}

__device__ __forceinline__ lg_range lg_slice(int V, int slices, int s) {
    lg_range r;
    r.whole = V / LG_VEC;
    r.rest = V % LG_VEC;
    const int n = r.whole + (r.rest != 0), each = lg_each(V, slices);
    r.v0 = min(n, s * each);
    r.v1 = min(n, r.v0 + each);
    return r;
}

// A thread's vectors of a slice: those of `turns` whole turns of the workgroup,
// one more where `more`, and the row's last one, part empty, where `part`.
//
// A walk up that another one down follows keeps the last HELD turns in LDS (64 bytes
// a thread: the rest of 160 KB when a CU is full of threads), read past the caches,
// which keep the others: a CU's share of the second-level cache is 128 KB.  2048 x
// 32000 fp16: gradient 62.8 us without, 57.9 with 32 bytes a thread, 54.5 with 64, 66.1
// with 128 (half the threads); its distillation 73, 66, 63, 82.
template <typename T, int TH>
struct lg_walk {
    static constexpr int AHEAD = 4;
    static constexpr int HELD = 64 / (int)sizeof(typename T::raw);
    static constexpr int HELD_BYTES = TH * 64;
    const typename T::bits *x;
    int v, turns, rest;     // v: the first vector
    bool more, part;
    uint4 *hold;            // (LDS)
    int held;               // turns there

    __device__ __forceinline__ lg_walk(const typename T::bits *row, const lg_range &r, void *room = nullptr) : x(row) {
        const int end = min(r.v1, r.whole);
        v = r.v0 + (int)threadIdx.x;
        turns = max(0, end - r.v0) / TH;
        const int last = v + turns * TH;
        more = last < end;
        part = (more ? last + TH : last) == r.whole && r.v1 > r.whole;
        rest = r.rest;
        hold = (uint4 *)room;
        held = room != nullptr ? min(turns, HELD) : 0;
    }
    __device__ __forceinline__ const typename T::bits *at(int turn) const {
        return x + (int64_t)(v + turn * TH) * LG_VEC;
    }
    // f(values, vector) of all, upwards
    template <typename F>
    __device__ __forceinline__ void up(F f) {
        int t = 0;
        const int cached = turns - held;
        for (; t + AHEAD <= cached; t += AHEAD) {
            typename T::raw raw[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                raw[i] = lg_load<T>(at(t + i));
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                float e[LG_VEC];
                lg_values<T>(raw[i], e);
                f(e, v + (t + i) * TH);
            }
        }
        for (; t < cached; ++t)
            one(t, f);
        if (held > 0) {
            typename T::raw raw[HELD];
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                raw[i] = lg_load_past<T>(at(t + min(i, held - 1)));
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                if (i >= held)
                    break;
                hold[i * TH + threadIdx.x] = __builtin_bit_cast(uint4, raw[i].a);
                if constexpr (sizeof(typename T::bits) == 4)
                    hold[(HELD + i) * TH + threadIdx.x] = __builtin_bit_cast(uint4, raw[i].b);
                float e[LG_VEC];
                lg_values<T>(raw[i], e);
                f(e, v + (t + i) * TH);
            }
        }
        if (more)
            one(turns, f);
        if (part) {
            float e[LG_VEC];
            lg_load_part<T>(at(turns + more), rest, e);
            f(e, v + (turns + more) * TH);
        }
    }
    template <typename F>
    __device__ __forceinline__ void one(int t, F f) {
        float e[LG_VEC];
        lg_values<T>(lg_load<T>(at(t)), e);
        f(e, v + t * TH);
    }
    // out = f(values, vector) of all, downwards: what was read last is still in
    // the caches.  A thread writes what it has read itself, so `out` may be x.
    // The stores leave the caches to what will be read again.
    template <typename F>
    __device__ __forceinline__ void down(typename T::bits *out, F f) {
        if (part) {
            float e[LG_VEC];
            const int64_t at_ = (int64_t)(v + (turns + more) * TH) * LG_VEC;
            lg_load_part<T>(x + at_, rest, e);
            f(e, v + (turns + more) * TH);
            lg_store_part<T>(out + at_, rest, e);
        }
        if (more)
            back(out, turns, f);
        int t = turns;
        if (held > 0) {
#pragma unroll
            for (int i = HELD - 1; i >= 0; --i) {
                if (i >= held)
                    continue;
                --t;
                typename T::raw raw;
                raw.a = __builtin_bit_cast(lg_u32x4, hold[i * TH + threadIdx.x]);
                if constexpr (sizeof(typename T::bits) == 4)
                    raw.b = __builtin_bit_cast(lg_u32x4, hold[(HELD + i) * TH + threadIdx.x]);
                float e[LG_VEC];
                lg_values<T>(raw, e);
                f(e, v + t * TH);
                lg_store<T>(out + (int64_t)(v + t * TH) * LG_VEC, e);
            }
        }
        for (; t >= AHEAD; t -= AHEAD) {
            typename T::raw raw[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                raw[i] = lg_load<T>(at(t - 1 - i));
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                float e[LG_VEC];
                lg_values<T>(raw[i], e);
                f(e, v + (t - 1 - i) * TH);
                lg_store<T>(out + (int64_t)(v + (t - 1 - i) * TH) * LG_VEC, e);
            }
        }
        for (; t > 0; --t)
            back(out, t - 1, f);
    }
    template <typename F>
    __device__ __forceinline__ void back(typename T::bits *out, int t, F f) {
        float e[LG_VEC];
        lg_values<T>(lg_load<T>(at(t)), e);
        f(e, v + t * TH);
        lg_store<T>(out + (int64_t)(v + t * TH) * LG_VEC, e);
    }
};

// The sums of the workgroup's vectors of a slice from v0 on, and, with TOP, the
// thread's largest entry and the first vector that holds it, and in `tops` (where
// given) the upper halves of the vectors' largest entries' keys.  `map` (LG_NAMED):
// a byte per vector.
template <typename T, int KIND, bool TOP, int TH, bool QUICK>
__device__ __forceinline__ void lg_stream(lg_walk<T, TH> &walk, float c, const uint8_t *map, int v0,
                                          lg_sums<QUICK> &s, float &best, int &where, uint16_t *tops = nullptr) {
    const float slack = QUICK ? LG_SLACK : LG_SLACK / c;
    walk.up([&](const float(&e)[LG_VEC], int at) __attribute__((always_inline)) {
        uint32_t named = 0;
        if constexpr (KIND == LG_NAMED)
            named = map[at - v0];
        const float top = lg_add<KIND>(s, e, c, slack, named);
        if (TOP) {
            if (tops != nullptr)
                tops[at - v0] = (uint16_t)(lg_ordered(top) >> 16);
            if (top > best) {
                best = top;
                where = at;
            }
        }
    });
}

// What the sums of a row say, whichever way they were formed.
struct lg_row {
    float m, S, b;      // reference; sum (LG_NAMED: of the entries not named), second sum
    bool quick;
    __device__ __forceinline__ float exponent(float x, float c) const {
        return quick ? lg_exponent<true>(x, m, c) : lg_exponent<false>(x, m, c);
    }
};

template <bool QUICK>
__device__ __forceinline__ lg_row lg_row_of(const lg_sums<QUICK> &t) {
    return {t.m, t.a, t.b, QUICK};
}

template <typename T, int TH>
__device__ __forceinline__ void lg_zero(typename T::bits *out, const lg_range &r) {
    const float zero[LG_VEC] = {};
    for (int v = r.v0 + (int)threadIdx.x; v < r.v1; v += TH) {
        if (v < r.whole)
            lg_store<T>(out + (int64_t)v * LG_VEC, zero);
        else
            lg_store_part<T>(out + (int64_t)v * LG_VEC, r.rest, zero);
    }
}

// One workgroup a unit.  A launch has less than 2^32 threads: more units take
// several.
template <typename F>
inline void lg_launches(lg_row_args &a, int64_t units, F launch) {
    constexpr int64_t MOST = 1 << 22;
    for (a.first = 0; a.first < units; a.first += MOST)
        launch((unsigned)(units - a.first < MOST ? units - a.first : MOST));
}

inline lg_row_args row_args(const void *x, int M, int V, int64_t stride, float temperature, int32_t *status) {
    lg_row_args a = {};
    a.x = x;
    a.stride = stride;
    a.M = M;
    a.V = V;
    a.c = (float)(1.4426950408889634 / (double)temperature);
    a.inv_t = (float)(1.0 / (double)temperature);
    a.status = status;
    return a;
}

// The slices' room in the workspace; one slice where it is too small.
inline void cut_rows(lg_row_args &a, int top, int slots, void *workspace, size_t bytes) {
    a.slices = logits_workspace_bytes(a.M, a.V, top, slots) > bytes ? 1 : logits_slices(a.M, a.V);
    const size_t units = (size_t)a.M * a.slices;
    a.sums = (float4 *)workspace;
    a.keys = (uint64_t *)((char *)workspace + units * 16u);
    a.named = (float *)((char *)workspace + units * (16u + 8u * (size_t)top));
}

}  // namespace rbq
