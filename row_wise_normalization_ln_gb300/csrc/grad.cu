// The global norm of a list of gradients, and clipping by it.
//
//   grad_sums    every CTA adds the squares of its share of the values and
//                leaves one fp64 partial sum.
//   grad_finish  one CTA adds the partial sums: the norm.
//   grad_scale   every CTA adds the partial sums itself (the same bits in
//                each) and multiplies its share by the coefficient.
//   grad_small   one CTA does it all for short lists, in one launch.
//
// The kernels stream: each value is read once per pass, which is all the
// arithmetic needs (bound: HBM; on one GB300 with a copy bandwidth of 6.8 TB/s,
// the norm of 1.6 GB in bf16 229 us, 7.0 TB/s; clipping 1 GB in fp32 into other
// buffers 467 to 476 us, 6.4 TB/s of its 3 GB: sums 150 us, scaling 306 to
// 315). The list is cut into units of one 16-byte access per thread of a CTA; CTA i of G takes
// the units [U i / G, U (i + 1) / G), so the shares differ by one unit at most
// however the sizes are mixed, and a share is a run of neighbouring addresses
// but for the steps between tensors. The scaling walks its shares from the
// end: what a CTA read last for the sums is what L2 still holds. Calls on a few
// MB are two launches of 3 to 6 us: 48 tensors of 45009 values, 6.5 MB, 12.6 us.
//
// The table of tensors travels in the kernel's argument block (up to 960
// tensors per launch), so nothing is copied to the device and a captured
// graph holds its own.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include <cuda_runtime_api.h>

#include "libnorm_grad.h"
#include "norm_args.h"
#include "norm_device.cuh"
#include "norm_kernels.cuh"

namespace libnorm {
namespace {

constexpr int kThreads = 256;          // of a CTA, and of a team of grad_small
constexpr int kSmallTeams = 4;         // of the one CTA of grad_small
constexpr int kSmallInFlight = 6;      // its accesses per thread
constexpr int kSmallUnits = kSmallTeams * kSmallInFlight;  // the longest list it takes: 96 KB
constexpr int kSmallTensors = 64;      // and the most tensors
constexpr int kUnroll = 8;             // accesses per thread in flight
constexpr int kUnitBytes = kThreads * 16;
constexpr int kCtasPerSm = 4;
constexpr int kMaxTable = 960;

template <int CAP>
struct GradTable {
    const void* data[CAP];
    void* out[CAP];
    int64_t numel[CAP];
    int64_t first[CAP + 1];  // first unit of each tensor; first[count]: all units
    uint8_t dtype[CAP];
    int32_t count;
};
static_assert(kThreads * kSmallTeams == 1024, "grad_small sums its 32 warps in one");
static_assert(sizeof(GradTable<kMaxTable>) + 64 <= 32764, "kernel arguments: 32764 bytes");

// A tensor's values: the few before the first 16-byte boundary, whole
// 16-byte accesses, the few after. Unit 0 takes the first few too, the last
// unit the last few.
struct Span {
    int64_t head, vecs, numel;
    int per;  // values per access
};
__device__ __forceinline__ Span span_of(const void* p, int64_t numel, int es) {
    Span s;
    s.per = 16 / es;
    s.numel = numel;
    s.head = min(numel, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / es));
    s.vecs = (numel - s.head) / s.per;
    return s;
}

// The tensor that unit `u` belongs to (tensors without values own no units).
template <int CAP>
__device__ __forceinline__ int tensor_of(const GradTable<CAP>& t, int64_t u) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float value_at(const void* p, int64_t i, int dtype) {
    if (dtype == NORM_F32) return static_cast<const float*>(p)[i];
    const uint32_t b = static_cast<const unsigned short*>(p)[i];
    return dtype == NORM_BF16 ? Bf16Pair::widen(b).x : F16Pair::widen(b).x;
}

__device__ __forceinline__ void put_at(void* p, int64_t i, int dtype, float v) {
    if (dtype == NORM_F32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<unsigned short*>(p)[i] =
            static_cast<unsigned short>(dtype == NORM_BF16 ? Bf16Pair::pack(v, 0.f) : F16Pair::pack(v, 0.f));
}

__device__ __forceinline__ uint32_t word(const uint4& r, int i) {
    return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
}

// fp32 sum of the squares of an access, added to acc (two chains).
template <int DT>
__device__ __forceinline__ float2 add_squares(const uint4& r, float2 acc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == NORM_F32) {
            const float v = __uint_as_float(word(r, i));
            if (i & 1) acc.y = fmaf(v, v, acc.y);
            else acc.x = fmaf(v, v, acc.x);
        } else {
            const float2 v = DT == NORM_BF16 ? Bf16Pair::widen(word(r, i)) : F16Pair::widen(word(r, i));
            acc = __ffma2_rn(v, v, acc);
        }
    }
    return acc;
}

// The squares of n accesses, kThreads apart from v on, in fp64: the values
// are read again, so that the usual path holds no registers for this one.
template <int DT>
__device__ __noinline__ double exact_squares(const uint4* v, int n) {
    double s = 0.0;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        const uint4 r = v[k * kThreads];
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = word(r, i);
            if constexpr (DT == NORM_F32) {
                const double x = __uint_as_float(w);
                s = fma(x, x, s);
            } else {
                const float2 p = DT == NORM_BF16 ? Bf16Pair::widen(w) : F16Pair::widen(w);
                s = fma(static_cast<double>(p.x), static_cast<double>(p.x), s);
                s = fma(static_cast<double>(p.y), static_cast<double>(p.y), s);
            }
        }
    }
    return s;
}

// Whether fp32 squares may have left the range: the sum is not finite or near
// the end of the range, or so small that squares may have been lost below
// fp32's smallest values (which is fine where every value is 0). Otherwise
// what a lost square was worth is below 2^-60 of the sum.
constexpr float kSmallSum = 8.27180613e-25f;  // 2^-80
constexpr float kLargeSum = 1.32922800e36f;   // 2^120
__device__ __forceinline__ bool in_range(float s) { return s >= kSmallSum && s <= kLargeSum; }

// A thread's sum: fp32 sums in range are added as an unevaluated pair with
// the error of each addition kept (Knuth's two-sum), 46 bits or more, and the
// rest in fp64, which stays 0 in the usual case. (The fp64 unit is a
// sixty-fourth of the fp32 ones: fp64 additions across the lanes of 32 warps
// per SM were a microsecond at the end of every launch.)
struct Sum {
    float hi = 0.f, lo = 0.f;
    double far = 0.0;

    __device__ __forceinline__ void pair(float h, float l) {
        const float t = hi + h, b = t - hi;
        lo += ((hi - (t - b)) + (h - b)) + l;
        hi = t;
    }
    __device__ __forceinline__ void add(float s) {
        pair(s, 0.f);
        if (hi > kLargeSum) {
            far += static_cast<double>(hi) + static_cast<double>(lo);
            hi = lo = 0.f;
        }
    }
    __device__ __forceinline__ void add_square(float v) {
        const float s = v * v;
        if (in_range(s)) add(s);
        else far = fma(static_cast<double>(v), static_cast<double>(v), far);
    }
};

// Adds the squares of the n accesses r (the rest zero), kThreads apart from v
// on.
// (Accesses that a thread does not have are set, not skipped: a register that
// is written under a predicate alone stays live through the whole loop, which
// tripled the registers.)
template <int DT>
__device__ __forceinline__ void squares(const uint4 (&r)[kUnroll], int n, const uint4* v, Sum& sum) {
    float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        if (k & 1) b = add_squares<DT>(r[k], b);
        else a = add_squares<DT>(r[k], a);
    }
    const float s = (a.x + a.y) + (b.x + b.y);
    if (in_range(s)) {
        sum.add(s);
        return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
        any |= r[k].x | r[k].y | r[k].z | r[k].w;
    if (any != 0) sum.far += exact_squares<DT>(v, n);
}

__device__ __forceinline__ double warp_sum(double v) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFullMask, v, off);
    return v;
}

// Sum over a CTA, in thread 0 (elsewhere undefined).
__device__ __forceinline__ double cta_sum(Sum v, double* part) {
    double w;
    if (__any_sync(kFullMask, v.far != 0.0)) {  // (NaN too)
        w = warp_sum(v.far + (static_cast<double>(v.hi) + static_cast<double>(v.lo)));
    } else {
        for (int off = 16; off > 0; off >>= 1) {
            const float h = __shfl_xor_sync(kFullMask, v.hi, off), l = __shfl_xor_sync(kFullMask, v.lo, off);
            v.pair(h, l);
        }
        w = static_cast<double>(v.hi) + static_cast<double>(v.lo);
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = w;
    __syncthreads();
    if (threadIdx.x != 0) return 0.0;
    static_assert(kThreads / 32 == 8, "eight partial sums");
    return ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
}

// sqrt(s) by one Newton step in fp64 from fp32's root (48 bits or more):
// the device's fp64 unit is a sixty-fourth of its fp32 ones, and its root and
// division took longer than a short list's memory.
__device__ __forceinline__ double root(double s) {
    if (!(s > 1e-30 && s < 1e30)) return sqrt(s);  // outside fp32's reach: rare
    const float r = sqrtf(static_cast<float>(s));
    const double y = r;
    return fma(fma(-y, y, s), static_cast<double>(0.5f / r), y);
}

// The coefficient of a norm, 1 at most, rounded once; NaN from a NaN norm.
__device__ __forceinline__ float coef_of(float max_norm, double norm) {
    const double d = norm + 1e-6, m = max_norm;
    double c;
    if (d < 1e30) {
        const float r = 1.f / static_cast<float>(d);
        const double c0 = m * static_cast<double>(r);
        c = fma(fma(-c0, d, m), static_cast<double>(r), c0);
    } else {  // infinite, NaN or beyond the reach of fp32's reciprocal
        c = m / d;
    }
    return c > 1.0 ? 1.f : static_cast<float>(c);
}

// How many of the next kUnroll accesses, kThreads apart, there are for a
// thread with `left` accesses from its first one to the tensor's end, in
// `units` units.
__device__ __forceinline__ int accesses(int64_t left, int64_t units) {
    const int64_t n = left <= 0 ? 0 : min(units, (left + kThreads - 1) / kThreads);
    return n < kUnroll ? static_cast<int>(n) : kUnroll;
}

// The units [u, stop) of one tensor: squares of this thread's values.
template <int DT>
__device__ __forceinline__ void piece_squares(const void* p, int64_t numel, int64_t u, int64_t stop, int64_t units, int tid,
                                              Sum& sum) {
    const Span s = span_of(p, numel, DT == NORM_F32 ? 4 : 2);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + s.head * (DT == NORM_F32 ? 4 : 2));
    if (u == 0 && tid < s.head) sum.add_square(value_at(p, tid, DT));
    const int64_t tail = s.head + s.vecs * s.per;
    if (stop == units && tail + tid < numel) sum.add_square(value_at(p, tail + tid, DT));
#pragma unroll 1
    for (; u < stop; u += kUnroll) {
        const uint4* at = v + u * kThreads + tid;
        const int n = accesses(s.vecs - u * kThreads - tid, stop - u);
        uint4 r[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            r[k] = k < n ? at[k * kThreads] : make_uint4(0, 0, 0, 0);
        if (n > 0) squares<DT>(r, n, at, sum);
    }
}

// Share i of n of the list: the sum of squares of this thread's values.
template <int CAP>
__device__ __forceinline__ Sum share_squares(const GradTable<CAP>& t, int64_t i, int64_t n, int tid) {
    const int64_t all = t.first[t.count];
    int64_t u = all * i / n;
    const int64_t end = all * (i + 1) / n;
    Sum sum;
    if (u < end) {
#pragma unroll 1
        for (int k = tensor_of(t, u); u < end; ++k) {
            const int64_t first = t.first[k], units = t.first[k + 1] - first;
            if (units == 0) continue;
            const int64_t a = u - first, b = min(units, end - first);
            const void* p = t.data[k];
            const int dt = t.dtype[k];
            if (dt == NORM_F32) piece_squares<NORM_F32>(p, t.numel[k], a, b, units, tid, sum);
            else if (dt == NORM_BF16) piece_squares<NORM_BF16>(p, t.numel[k], a, b, units, tid, sum);
            else piece_squares<NORM_F16>(p, t.numel[k], a, b, units, tid, sum);
            u = first + b;
        }
    }
    return sum;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_sums(const __grid_constant__ GradTable<CAP> t,
                                                                  double* partial) {
    __shared__ double part[kThreads / 32];
    grid_release();
    grid_wait();
    const double sum = cta_sum(share_squares(t, blockIdx.x, gridDim.x, threadIdx.x), part);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The sum of the n partial sums, in every lane of the one warp that calls it.
__device__ __forceinline__ double sum_partials(const double* partial, int64_t n) {
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += 32) s += partial[i];
    return warp_sum(s);
}

__global__ void __launch_bounds__(32) grad_finish(const double* partial, int64_t n, float* norm) {
    grid_release();
    grid_wait();
    const double s = sum_partials(partial, n);
    if (threadIdx.x == 0) *norm = static_cast<float>(root(s));
}

template <int DT>
__device__ __forceinline__ uint4 scaled(const uint4& r, float coef) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == NORM_F32) {
            o[i] = __float_as_uint(__uint_as_float(word(r, i)) * coef);
        } else {
            const float2 v = __fmul2_rn(DT == NORM_BF16 ? Bf16Pair::widen(word(r, i)) : F16Pair::widen(word(r, i)),
                                        f2_splat(coef));
            o[i] = DT == NORM_BF16 ? Bf16Pair::pack(v.x, v.y) : F16Pair::pack(v.x, v.y);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A thread's value of the first few and of the last few (0 where it has
// none): read before the whole accesses, used after them, so that a piece
// waits for memory once.
template <int DT>
struct Edges {
    float head = 0.f, tail = 0.f;
    int first, last;  // how many there are
    __device__ __forceinline__ Edges(const void* p, int64_t numel, int64_t head_values, int64_t tail_at, bool has_head,
                                     bool has_tail, int tid)
        : first(has_head ? static_cast<int>(head_values) : 0), last(has_tail ? static_cast<int>(numel - tail_at) : 0) {
        if (tid < first) head = value_at(p, tid, DT);
        if (tid < last) tail = value_at(p, numel - last + tid, DT);
    }
    __device__ __forceinline__ void put(void* out, int64_t numel, float coef, int tid) const {
        if (tid < first) put_at(out, tid, DT, head * coef);
        if (tid < last) put_at(out, numel - last + tid, DT, tail * coef);
    }
};

// The 16 bytes from byte `by` of (a, b) on.
__device__ __forceinline__ uint4 straddled(const uint4& a, const uint4& b, int by) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = by & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = by & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (by & 2) * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The units [u, stop) of one tensor, from the last to the first.
template <int DT>
__device__ __forceinline__ void piece_scale(const void* p, void* out, int64_t numel, int64_t u, int64_t stop,
                                            int64_t units, float coef, int tid) {
    constexpr int es = DT == NORM_F32 ? 4 : 2;
    const uintptr_t from = reinterpret_cast<uintptr_t>(p), to = reinterpret_cast<uintptr_t>(out);
    if (((from ^ to) & 15) != 0) {
        // out lies at another offset within 16 bytes: whole accesses of out,
        // each from the two accesses of p that it straddles, where both lie
        // within the tensor
        Span s = span_of(out, numel, es);
        if (s.head < numel && ((from + s.head * es) & ~uintptr_t(15)) < from) s.head += s.per;
        s.head = min(s.head, numel);
        const uintptr_t base = (from + s.head * es) & ~uintptr_t(15);
        const int by = static_cast<int>((from + s.head * es) & 15);
        s.vecs = max(int64_t(0), static_cast<int64_t>(from + numel * es - base) / 16 - 1);
        const Edges<DT> edges(p, numel, s.head, s.head + s.vecs * s.per, u == 0, stop == units, tid);
        const uint4* v = reinterpret_cast<const uint4*>(base);
        uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(out) + s.head * es);
        constexpr int kPairs = 3;  // (4 spill)
#pragma unroll 1
        for (int64_t e = stop; e > u; e -= kPairs) {
            const int64_t f = max(u, e - kPairs);
            const int64_t i = f * kThreads + tid;
            const int n = accesses(s.vecs - i, e - f);
            uint4 a[kPairs], b[kPairs];
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                a[k] = k < n ? v[i + k * kThreads] : make_uint4(0, 0, 0, 0);
                b[k] = k < n ? v[i + k * kThreads + 1] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < kPairs; ++k)
                if (k < n) o[i + k * kThreads] = scaled<DT>(straddled(a[k], b[k], by), coef);
        }
        edges.put(out, numel, coef, tid);
        return;
    }
    const Span s = span_of(p, numel, es);
    const Edges<DT> edges(p, numel, s.head, s.head + s.vecs * s.per, u == 0, stop == units, tid);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + s.head * es);
    uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(out) + s.head * es);
#pragma unroll 1
    for (int64_t e = stop; e > u; e -= kUnroll) {
        const int64_t f = max(u, e - kUnroll);
        const int64_t i = f * kThreads + tid;
        const int n = accesses(s.vecs - i, e - f);
        uint4 r[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            r[k] = k < n ? v[i + k * kThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (k < n) o[i + k * kThreads] = scaled<DT>(r[k], coef);
    }
    edges.put(out, numel, coef, tid);
}

// Share i of n of the list, from its end: times coef.
template <int CAP>
__device__ __forceinline__ void share_scale(const GradTable<CAP>& t, int64_t i, int64_t n, float coef, int tid) {
    const int64_t all = t.first[t.count];
    const int64_t begin = all * i / n;
    int64_t e = all * (i + 1) / n;
    if (begin >= e) return;
#pragma unroll 1
    for (int k = tensor_of(t, e - 1); e > begin; --k) {
        const int64_t first = t.first[k], units = t.first[k + 1] - first;
        if (units == 0) continue;
        const int64_t a = max(begin - first, int64_t(0)), b = e - first;
        const void* p = t.data[k];
        void* o = t.out[k];
        // x * 1 is x: in place there is nothing to do
        if (!(coef == 1.f && p == o)) {
            const int dt = t.dtype[k];
            if (dt == NORM_F32) piece_scale<NORM_F32>(p, o, t.numel[k], a, b, units, coef, tid);
            else if (dt == NORM_BF16) piece_scale<NORM_BF16>(p, o, t.numel[k], a, b, units, coef, tid);
            else piece_scale<NORM_F16>(p, o, t.numel[k], a, b, units, coef, tid);
        }
        e = first + a;
    }
}

// norm: written by the first launch's first CTA only (null elsewhere).
template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_scale(const __grid_constant__ GradTable<CAP> t,
                                                                   const double* partial, int64_t n, float max_norm,
                                                                   float* norm) {
    __shared__ float coef;
    grid_release();
    grid_wait();
    if (threadIdx.x < 32) {  // (one warp: fp64 is scarce)
        const double total = root(sum_partials(partial, n));
        if (threadIdx.x == 0) {
            coef = coef_of(max_norm, total);
            if (norm != nullptr && blockIdx.x == 0) *norm = static_cast<float>(total);
        }
    }
    __syncthreads();
    share_scale(t, blockIdx.x, gridDim.x, coef, threadIdx.x);
}

// ------------------------------------------------------------ short lists
// One access of a tensor: values [j * per, (j + 1) * per), zeros past the end.
template <int DT>
__device__ __forceinline__ uint4 load_slot(const void* p, int64_t j, int64_t numel) {
    constexpr int per = DT == NORM_F32 ? 4 : 8;
    const int64_t at = j * per, left = numel - at;
    if (left >= per && (reinterpret_cast<uintptr_t>(p) & 15) == 0) return static_cast<const uint4*>(p)[j];
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < per; ++i)
        if (i < left) {
            if constexpr (DT == NORM_F32) w[i] = static_cast<const uint32_t*>(p)[at + i];
            else w[i / 2] |= uint32_t(static_cast<const unsigned short*>(p)[at + i]) << (16 * (i & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT>
__device__ __forceinline__ void store_slot(void* p, int64_t j, int64_t numel, const uint4& r) {
    constexpr int per = DT == NORM_F32 ? 4 : 8;
    const int64_t at = j * per, left = numel - at;
    if (left >= per && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        static_cast<uint4*>(p)[j] = r;
        return;
    }
#pragma unroll
    for (int i = 0; i < per; ++i)
        if (i < left) {
            if constexpr (DT == NORM_F32) static_cast<uint32_t*>(p)[at + i] = word(r, i);
            else static_cast<unsigned short*>(p)[at + i] = static_cast<unsigned short>(word(r, i / 2) >> (16 * (i & 1)));
        }
}
template <int DT>
__device__ __forceinline__ float slot_squares(const uint4& r) {
    const float2 a = add_squares<DT>(r, make_float2(0.f, 0.f));
    return a.x + a.y;
}

// (Bound: launch and one load's latency. 24 tensors of 1024 fp32 values 3.8 us,
// one of 512 2.0.)
// The whole of a list of at most kSmallTensors tensors and kSmallUnits units
// in one CTA and one launch: the norm, and with CLIP the scaling. Its teams
// take the units in turn, all of them in flight at once and kept in registers,
// so that the list waits for memory once.
template <bool CLIP>
__global__ void __launch_bounds__(kThreads* kSmallTeams) grad_small(const __grid_constant__ GradTable<kSmallTensors> t,
                                                                    float max_norm, float* norm) {
    __shared__ double part[kThreads * kSmallTeams / 32];
    __shared__ float coefficient;
    __shared__ int ends[kSmallTensors];  // the unit after each tensor's last
    grid_release();
    const int team = threadIdx.x / kThreads, tid = threadIdx.x & (kThreads - 1), lane = threadIdx.x & 31;
    if (threadIdx.x < kSmallTensors)
        ends[threadIdx.x] = threadIdx.x < t.count ? static_cast<int>(t.first[threadIdx.x + 1]) : 1 << 30;
    __syncthreads();
    const int all = static_cast<int>(t.first[t.count]);
    // the tensor of a unit: how many end at or before it
    auto tensor = [&](int u) {
        int i = 0;
#pragma unroll
        for (int k = 0; k < kSmallTensors; k += 32) i += __popc(__ballot_sync(kFullMask, ends[k + lane] <= u));
        return i;
    };
    // this thread's access within a unit's tensor
    auto access = [&](int i, int u) { return int64_t(u - (i > 0 ? ends[i - 1] : 0)) * kThreads + tid; };
    auto load = [&](int i, int64_t j) {
        const int dt = t.dtype[i];
        return dt == NORM_F32    ? load_slot<NORM_F32>(t.data[i], j, t.numel[i])
               : dt == NORM_BF16 ? load_slot<NORM_BF16>(t.data[i], j, t.numel[i])
                                 : load_slot<NORM_F16>(t.data[i], j, t.numel[i]);
    };
    grid_wait();
    uint4 r[kSmallInFlight];
#pragma unroll
    for (int k = 0; k < kSmallInFlight; ++k) {
        const int u = team + k * kSmallTeams;
        r[k] = make_uint4(0, 0, 0, 0);
        if (u < all) {
            const int i = tensor(u);
            r[k] = load(i, access(i, u));
        }
    }
    // fp32 over a warp's values (32 per lane at most), fp64 beyond: the whole
    // warp goes to fp64 where a lane's or the warp's sum may have left fp32's
    // range.
    float v = 0.f;
    bool lost = false;
#pragma unroll
    for (int k = 0; k < kSmallInFlight; ++k) {
        const int u = team + k * kSmallTeams;
        if (u >= all) break;
        const int dt = t.dtype[tensor(u)];
        const float s = dt == NORM_F32    ? slot_squares<NORM_F32>(r[k])
                        : dt == NORM_BF16 ? slot_squares<NORM_BF16>(r[k])
                                          : slot_squares<NORM_F16>(r[k]);
        lost |= !(s >= kSmallSum) && (r[k].x | r[k].y | r[k].z | r[k].w) != 0;
        v += s;
    }
    v = group_sum(v, 32);
    double sum = static_cast<double>(v);
    if (__any_sync(kFullMask, lost) || !(v <= 3.0e38f)) {
        double d = 0.0;
#pragma unroll 1
        for (int u = team; u < all; u += kSmallTeams) {
            const int i = tensor(u);
            const uint4 w = load(i, access(i, u));
            d += t.dtype[i] == NORM_F32    ? exact_squares<NORM_F32>(&w, 1)
                 : t.dtype[i] == NORM_BF16 ? exact_squares<NORM_BF16>(&w, 1)
                                           : exact_squares<NORM_F16>(&w, 1);
        }
        sum = warp_sum(d);
    }
    if (lane == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        const double total = root(warp_sum(part[lane]));
        if (threadIdx.x == 0) {
            *norm = static_cast<float>(total);
            if constexpr (CLIP) coefficient = coef_of(max_norm, total);
        }
    }
    if constexpr (CLIP) {
        __syncthreads();
        const float coef = coefficient;
#pragma unroll
        for (int k = 0; k < kSmallInFlight; ++k) {
            const int u = team + k * kSmallTeams;
            if (u >= all) break;
            const int i = tensor(u);
            if (coef == 1.f && t.data[i] == t.out[i]) continue;  // x * 1 is x
            const int64_t j = access(i, u);
            const int dt = t.dtype[i];
            if (dt == NORM_F32) store_slot<NORM_F32>(t.out[i], j, t.numel[i], scaled<NORM_F32>(r[k], coef));
            else if (dt == NORM_BF16) store_slot<NORM_BF16>(t.out[i], j, t.numel[i], scaled<NORM_BF16>(r[k], coef));
            else store_slot<NORM_F16>(t.out[i], j, t.numel[i], scaled<NORM_F16>(r[k], coef));
        }
    }
}

cudaError_t launch(const void* fn, int64_t grid, int threads, cudaStream_t stream, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int elem_size(int dtype) { return dtype == NORM_F32 ? 4 : 2; }
int64_t launches_of(int64_t count) { return std::max<int64_t>(1, ceil_div(count, kMaxTable)); }

template <int CAP>
void fill(GradTable<CAP>* t, const norm_tensor* ts, int64_t n) {
    int64_t u = 0;
    for (int64_t i = 0; i < n; ++i) {
        t->data[i] = ts[i].data;
        t->out[i] = ts[i].out;
        t->numel[i] = ts[i].numel;
        t->dtype[i] = static_cast<uint8_t>(ts[i].dtype);
        t->first[i] = u;
        u += ceil_div(ts[i].numel * elem_size(ts[i].dtype), kUnitBytes);
    }
    t->first[n] = u;
    t->count = static_cast<int32_t>(n);
}

// One table's pass of the sums (partial sums from `partial` on) or, with
// `clip`, of the scaling by all `n` partial sums.
template <int CAP>
cudaError_t pass(const norm_tensor* ts, int64_t count, bool clip, int64_t ctas, double* partial, int64_t n,
                 float max_norm, float* norm, cudaStream_t stream) {
    GradTable<CAP> t;
    fill(&t, ts, count);
    if (!clip) {
        void* args[] = {&t, &partial};
        return launch(reinterpret_cast<const void*>(grad_sums<CAP>), ctas, kThreads, stream, args);
    }
    const double* src = partial;
    void* args[] = {&t, &src, &n, &max_norm, &norm};
    return launch(reinterpret_cast<const void*>(grad_scale<CAP>), ctas, kThreads, stream, args);
}

cudaError_t any_pass(const norm_tensor* ts, int64_t count, bool clip, int64_t ctas, double* partial, int64_t n,
                     float max_norm, float* norm, cudaStream_t stream) {
    return count <= 64 ? pass<64>(ts, count, clip, ctas, partial, n, max_norm, norm, stream)
                       : pass<kMaxTable>(ts, count, clip, ctas, partial, n, max_norm, norm, stream);
}

cudaError_t small(const norm_tensor* ts, int64_t count, bool clip, float max_norm, float* norm, cudaStream_t stream) {
    GradTable<kSmallTensors> t;
    fill(&t, ts, count);
    void* args[] = {&t, &max_norm, &norm};
    const void* fn = clip ? reinterpret_cast<const void*>(grad_small<true>) : reinterpret_cast<const void*>(grad_small<false>);
    return launch(fn, 1, kThreads * kSmallTeams, stream, args);
}

int64_t units_of(const norm_tensor* ts, int64_t count) {
    int64_t u = 0;
    for (int64_t i = 0; i < count; ++i) u += ceil_div(ts[i].numel * elem_size(ts[i].dtype), kUnitBytes);
    return u;
}

// Lists that grad_small takes.
bool is_short(const norm_tensor* ts, int64_t count) {
    return count <= kSmallTensors && units_of(ts, count) <= kSmallUnits;
}

norm_status check_tensors(const norm_tensor* ts, int64_t count, bool clip) {
    if (count < 0 || count > (int64_t(1) << 24) || (count > 0 && !ts)) return NORM_ERR_ARG;
    for (int64_t i = 0; i < count; ++i) {
        const norm_tensor& t = ts[i];
        if (t.dtype != NORM_F32 && t.dtype != NORM_BF16 && t.dtype != NORM_F16) return NORM_ERR_DTYPE;
        if (t.numel < 0 || t.numel >= (int64_t(1) << 46)) return NORM_ERR_ARG;
        if (t.numel == 0) continue;
        const uintptr_t mask = static_cast<uintptr_t>(elem_size(t.dtype) - 1);
        if (!t.data || (reinterpret_cast<uintptr_t>(t.data) & mask)) return NORM_ERR_ARG;
        if (clip && (!t.out || (reinterpret_cast<uintptr_t>(t.out) & mask))) return NORM_ERR_ARG;
    }
    return NORM_OK;
}

// No output may overlap another tensor's output or input, or its own input
// other than exactly; the norm is an output of its own (grad_scale writes it
// while other CTAs read and write).
norm_status check_apart(const norm_tensor* ts, int64_t count, const float* norm) {
    struct Piece {
        uintptr_t lo, hi;
        bool write;
    };
    std::unique_ptr<Piece[]> p(new (std::nothrow) Piece[2 * static_cast<size_t>(count) + 1]);
    if (!p) return NORM_ERR_ARG;
    size_t n = 0;
    const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
    p[n++] = Piece{at, at + sizeof *norm, true};
    for (int64_t i = 0; i < count; ++i) {
        const uintptr_t bytes = static_cast<uintptr_t>(ts[i].numel) * elem_size(ts[i].dtype);
        if (bytes == 0) continue;
        const uintptr_t d = reinterpret_cast<uintptr_t>(ts[i].data), o = reinterpret_cast<uintptr_t>(ts[i].out);
        p[n++] = Piece{o, o + bytes, true};
        if (d != o) p[n++] = Piece{d, d + bytes, false};
    }
    std::sort(p.get(), p.get() + n, [](const Piece& a, const Piece& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;
    for (size_t i = 0; i < n; ++i) {
        if (p[i].lo < (p[i].write ? any : written)) return NORM_ERR_ARG;
        any = std::max(any, p[i].hi);
        if (p[i].write) written = std::max(written, p[i].hi);
    }
    return NORM_OK;
}

norm_status run(const norm_tensor* ts, int64_t count, bool clip, float max_norm, float* norm, void* ws,
                size_t ws_bytes, cudaStream_t stream) {
    norm_status st = check_tensors(ts, count, clip);
    if (st != NORM_OK) return st;
    if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u)) return NORM_ERR_ARG;
    if (clip && (!std::isfinite(max_norm) || max_norm < 0.f)) return NORM_ERR_ARG;
    const bool shortlist = is_short(ts, count);
    if (!shortlist && (!ws || (reinterpret_cast<uintptr_t>(ws) & 7u))) return NORM_ERR_ARG;
    if (clip && (st = check_apart(ts, count, norm)) != NORM_OK) return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    static std::atomic<int> cache[64];
    if (e == cudaSuccess && dev >= 0 && dev < 64) sms = cache[dev].load(std::memory_order_relaxed);
    if (e == cudaSuccess && sms <= 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && dev >= 0 && dev < 64) cache[dev].store(sms, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) {
        note_cuda_error(static_cast<int>(e));
        return NORM_ERR_CUDA;
    }
    size_t need = 0;
    grad_workspace_bytes(ts, count, sms, &need);
    if (ws_bytes < need) return NORM_ERR_ARG;
    // Short lists: one launch and no workspace. Tensors of 512 fp32 values,
    // norm / clipping in us against the two launches: 24 of them 4.0 / 6.3 to
    // 4.2 / 6.5, 32 of them 4.7 / 7.5 to 4.2 / 6.5.
    if (shortlist) {
        e = small(ts, count, clip, max_norm, norm, stream);
        if (e == cudaSuccess) return NORM_OK;
        note_cuda_error(static_cast<int>(e));
        return NORM_ERR_CUDA;
    }
    double* partial = static_cast<double*>(ws);
    // As many CTAs on each SM as let one read its share in one step of kUnroll
    // units, kCtasPerSm at most: grad_clip of 24 fp32 and 24 bf16 tensors of
    // 45009 values 12.6 us with the 304 of this rule, 14.0 with 152 or 608;
    // of 16 MB in one tensor 14.3 with 608, 17.6 with 456.
    const auto ctas_of = [&](int64_t units) {
        const int64_t per_sm = ceil_div(units, int64_t(sms) * kUnroll);
        return std::min(units, sms * std::max<int64_t>(1, std::min<int64_t>(kCtasPerSm, per_sm)));
    };
    int64_t n = 0;
    for (int64_t at = 0; at < count; at += kMaxTable) {
        const int64_t k = std::min<int64_t>(kMaxTable, count - at);
        const int64_t units = units_of(ts + at, k);
        const int64_t ctas = ctas_of(units);
        if (ctas == 0) continue;
        e = any_pass(ts + at, k, false, ctas, partial + n, 0, 0.f, nullptr, stream);
        if (e != cudaSuccess) break;
        n += ctas;
    }
    if (e == cudaSuccess && !clip) {
        const double* src = partial;
        void* args[] = {&src, &n, &norm};
        e = launch(reinterpret_cast<const void*>(grad_finish), 1, 32, stream, args);
    }
    for (int64_t at = 0; e == cudaSuccess && clip && at < std::max<int64_t>(count, 1); at += kMaxTable) {
        const int64_t k = std::min<int64_t>(kMaxTable, count - at);
        e = any_pass(ts + at, k, true, std::max<int64_t>(1, ctas_of(units_of(ts + at, k))), partial, n, max_norm,
                     at == 0 ? norm : nullptr, stream);
    }
    if (e != cudaSuccess) {
        note_cuda_error(static_cast<int>(e));
        return NORM_ERR_CUDA;
    }
    return NORM_OK;
}

}  // namespace
}  // namespace libnorm

extern "C" {

norm_status grad_norm(const norm_tensor* tensors, int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream) {
    return libnorm::run(tensors, count, false, 0.f, norm, workspace, workspace_bytes, stream);
}

norm_status grad_clip(const norm_tensor* tensors, int64_t count, float max_norm, float* norm, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
    return libnorm::run(tensors, count, true, max_norm, norm, workspace, workspace_bytes, stream);
}

norm_status grad_workspace_bytes(const norm_tensor* tensors, int64_t count, int num_sms, size_t* bytes) {
    const norm_status st = libnorm::check_tensors(tensors, count, false);
    if (st != NORM_OK) return st;
    if (!bytes || num_sms < 1) return NORM_ERR_ARG;
    *bytes = libnorm::is_short(tensors, count)
                 ? 0
                 : static_cast<size_t>(libnorm::launches_of(count)) * static_cast<size_t>(num_sms) * libnorm::kCtasPerSm * 8;
    return NORM_OK;
}

}  // extern "C"
