// The global norm of a list of gradients, and clipping by it.
//
//   grad_sums    every CTA adds the squares of its share of the values and
//                leaves one fp64 partial sum.
//   grad_finish  one CTA adds the partial sums: the norm.
//   grad_scale   every CTA adds the partial sums itself (the same bits in
//                each) and multiplies its share by the coefficient.
//
// Both kernels stream: each value is read once per kernel, which is all the
// arithmetic needs (bound: HBM). The list is cut into units of one 16-byte
// access per thread; CTA i takes the units [U i / G, U (i + 1) / G), so the
// shares differ by one unit at most however the sizes are mixed, and a share
// is a run of neighbouring addresses but for the steps between tensors. The
// scale kernel walks its shares from the end: what a CTA of the sums kernel
// read last is what L2 still holds.
//
// The table of tensors travels in the kernel's argument block (up to 960
// tensors per launch), so nothing is copied to the device and a captured
// graph holds its own.
#include <algorithm>
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

constexpr int kThreads = 256;
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

template <int DT>
__device__ __noinline__ double exact_squares(const uint4* r, int n) {
    double s = 0.0;
    for (int k = 0; k < n; ++k)
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = word(r[k], i);
            if constexpr (DT == NORM_F32) {
                const double v = __uint_as_float(w);
                s = fma(v, v, s);
            } else {
                const float2 p = DT == NORM_BF16 ? Bf16Pair::widen(w) : F16Pair::widen(w);
                const double x = p.x, y = p.y;
                s = fma(x, x, s);
                s = fma(y, y, s);
            }
        }
    return s;
}

// Whether fp32 squares may have left the range: the sum is not finite, or so
// small that squares may have been lost below fp32's smallest values (which
// is fine where every value is 0). Otherwise what a lost square was worth is
// below 2^-60 of the sum.
constexpr float kSmallSum = 8.27180613e-25f;  // 2^-80

template <int DT>
__device__ __forceinline__ double squares(const uint4 (&r)[kUnroll], int n) {
    float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
        if (k < n) {
            if (k & 1) b = add_squares<DT>(r[k], b);
            else a = add_squares<DT>(r[k], a);
        }
    const float s = (a.x + a.y) + (b.x + b.y);
    if (!(s >= kSmallSum && s <= 3.0e38f)) {
        uint32_t any = 0;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (k < n) any |= r[k].x | r[k].y | r[k].z | r[k].w;
        if (any != 0) {
            uint4 copy[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) copy[k] = r[k];
            return exact_squares<DT>(copy, n);
        }
    }
    return static_cast<double>(s);
}

__device__ __forceinline__ double warp_sum(double v) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFullMask, v, off);
    return v;
}

// Sum over the CTA, the same bits in every thread.
__device__ __forceinline__ double cta_sum(double v, double* part) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

// The units [u, stop) of one tensor: squares of this thread's values.
template <int DT>
__device__ __forceinline__ double piece_squares(const void* p, int64_t numel, int64_t u, int64_t stop, int64_t units) {
    const Span s = span_of(p, numel, DT == NORM_F32 ? 4 : 2);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + s.head * (DT == NORM_F32 ? 4 : 2));
    double sum = 0.0;
    if (u == 0 && static_cast<int64_t>(threadIdx.x) < s.head) {
        const double x = value_at(p, threadIdx.x, DT);
        sum = fma(x, x, sum);
    }
    const int64_t tail = s.head + s.vecs * s.per;
    if (stop == units && tail + static_cast<int64_t>(threadIdx.x) < numel) {
        const double x = value_at(p, tail + threadIdx.x, DT);
        sum = fma(x, x, sum);
    }
    for (; u < stop; u += kUnroll) {
        uint4 r[kUnroll];
        int n = 0;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t i = (u + k) * kThreads + threadIdx.x;
            if (u + k < stop && i < s.vecs) {
                r[k] = v[i];
                n = k + 1;
            }
        }
        if (n > 0) sum += squares<DT>(r, n);
    }
    return sum;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_sums(const __grid_constant__ GradTable<CAP> t, double* partial) {
    __shared__ double part[kThreads / 32];
    grid_release();
    grid_wait();
    const int64_t all = t.first[t.count];
    int64_t u = all * blockIdx.x / gridDim.x;
    const int64_t end = all * (blockIdx.x + 1ll) / gridDim.x;
    double sum = 0.0;
    if (u < end) {
        for (int i = tensor_of(t, u); u < end; ++i) {
            const int64_t first = t.first[i], units = t.first[i + 1] - first;
            if (units == 0) continue;
            const int64_t a = u - first, b = min(units, end - first);
            const void* p = t.data[i];
            const int dt = t.dtype[i];
            if (dt == NORM_F32) sum += piece_squares<NORM_F32>(p, t.numel[i], a, b, units);
            else if (dt == NORM_BF16) sum += piece_squares<NORM_BF16>(p, t.numel[i], a, b, units);
            else sum += piece_squares<NORM_F16>(p, t.numel[i], a, b, units);
            u = first + b;
        }
    }
    sum = cta_sum(sum, part);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__device__ __forceinline__ double sum_partials(const double* partial, int64_t n, double* part) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += partial[i];
    return cta_sum(s, part);
}

__global__ void __launch_bounds__(kThreads) grad_finish(const double* partial, int64_t n, float* norm) {
    __shared__ double part[kThreads / 32];
    grid_release();
    grid_wait();
    const double s = sum_partials(partial, n, part);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
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

// The units [u, stop) of one tensor, from the last to the first.
template <int DT>
__device__ __forceinline__ void piece_scale(const void* p, void* out, int64_t numel, int64_t u, int64_t stop,
                                            int64_t units, float coef) {
    constexpr int es = DT == NORM_F32 ? 4 : 2;
    const Span s = span_of(p, numel, es);
    const int64_t tail = s.head + s.vecs * s.per;
    if (u == 0 && static_cast<int64_t>(threadIdx.x) < s.head)
        put_at(out, threadIdx.x, DT, value_at(p, threadIdx.x, DT) * coef);
    if (stop == units && tail + static_cast<int64_t>(threadIdx.x) < numel)
        put_at(out, tail + threadIdx.x, DT, value_at(p, tail + threadIdx.x, DT) * coef);
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
        // out lies at another offset within 16 bytes: value by value
        const int64_t lo = s.head + min(s.vecs, u * kThreads) * s.per, hi = s.head + min(s.vecs, stop * kThreads) * s.per;
        for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) put_at(out, i, DT, value_at(p, i, DT) * coef);
        return;
    }
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + s.head * es);
    uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(out) + s.head * es);
    for (int64_t e = stop; e > u; e -= kUnroll) {
        uint4 r[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t i = (e - 1 - k) * kThreads + threadIdx.x;
            if (e - 1 - k >= u && i < s.vecs) r[k] = v[i];
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t i = (e - 1 - k) * kThreads + threadIdx.x;
            if (e - 1 - k >= u && i < s.vecs) o[i] = scaled<DT>(r[k], coef);
        }
    }
}

// norm: written by the first launch's first CTA only (null elsewhere).
template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_scale(const __grid_constant__ GradTable<CAP> t, const double* partial,
                                                       int64_t n, float max_norm, float* norm) {
    __shared__ double part[kThreads / 32];
    grid_release();
    grid_wait();
    const double total = sqrt(sum_partials(partial, n, part));
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
    // in fp64, rounded once; a NaN norm gives a NaN coefficient
    const double c = static_cast<double>(max_norm) / (total + 1e-6);
    const float coef = c > 1.0 ? 1.f : static_cast<float>(c);
    const int64_t all = t.first[t.count];
    const int64_t begin = all * blockIdx.x / gridDim.x;
    int64_t e = all * (blockIdx.x + 1ll) / gridDim.x;
    if (begin >= e) return;
    for (int i = tensor_of(t, e - 1); e > begin; --i) {
        const int64_t first = t.first[i], units = t.first[i + 1] - first;
        if (units == 0) continue;
        const int64_t a = max(begin - first, int64_t(0)), b = e - first;
        const void* p = t.data[i];
        void* o = t.out[i];
        // x * 1 is x: in place there is nothing to do
        if (!(coef == 1.f && p == o)) {
            const int dt = t.dtype[i];
            if (dt == NORM_F32) piece_scale<NORM_F32>(p, o, t.numel[i], a, b, units, coef);
            else if (dt == NORM_BF16) piece_scale<NORM_BF16>(p, o, t.numel[i], a, b, units, coef);
            else piece_scale<NORM_F16>(p, o, t.numel[i], a, b, units, coef);
        }
        e = first + a;
    }
}

cudaError_t launch(const void* fn, int64_t grid, cudaStream_t stream, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
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
        return launch(reinterpret_cast<const void*>(grad_sums<CAP>), ctas, stream, args);
    }
    const int64_t grid = std::max<int64_t>(1, std::min(ctas, t.first[count]));
    const double* src = partial;
    void* args[] = {&t, &src, &n, &max_norm, &norm};
    return launch(reinterpret_cast<const void*>(grad_scale<CAP>), grid, stream, args);
}

cudaError_t any_pass(const norm_tensor* ts, int64_t count, bool clip, int64_t ctas, double* partial, int64_t n,
                     float max_norm, float* norm, cudaStream_t stream) {
    return count <= 64 ? pass<64>(ts, count, clip, ctas, partial, n, max_norm, norm, stream)
                       : pass<kMaxTable>(ts, count, clip, ctas, partial, n, max_norm, norm, stream);
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
// other than exactly.
norm_status check_apart(const norm_tensor* ts, int64_t count) {
    struct Piece {
        uintptr_t lo, hi;
        bool write;
    };
    std::unique_ptr<Piece[]> p(new (std::nothrow) Piece[2 * static_cast<size_t>(count) + 1]);
    if (!p) return NORM_ERR_ARG;
    size_t n = 0;
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
    if (!norm || (clip && (!std::isfinite(max_norm) || max_norm < 0.f))) return NORM_ERR_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 7u)) return NORM_ERR_ARG;
    if (clip && (st = check_apart(ts, count)) != NORM_OK) return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
        note_cuda_error(static_cast<int>(e));
        return NORM_ERR_CUDA;
    }
    size_t need = 0;
    grad_workspace_bytes(count, sms, &need);
    if (ws_bytes < need) return NORM_ERR_ARG;
    double* partial = static_cast<double*>(ws);
    const int64_t most = int64_t(sms) * kCtasPerSm;
    int64_t n = 0;
    for (int64_t at = 0; at < count; at += kMaxTable) {
        const int64_t k = std::min<int64_t>(kMaxTable, count - at);
        int64_t units = 0;
        for (int64_t i = at; i < at + k; ++i) units += ceil_div(ts[i].numel * elem_size(ts[i].dtype), kUnitBytes);
        const int64_t ctas = std::min(most, units);
        if (ctas == 0) continue;
        e = any_pass(ts + at, k, false, ctas, partial + n, 0, 0.f, nullptr, stream);
        if (e != cudaSuccess) break;
        n += ctas;
    }
    if (e == cudaSuccess && !clip) {
        const double* src = partial;
        void* args[] = {&src, &n, &norm};
        e = launch(reinterpret_cast<const void*>(grad_finish), 1, stream, args);
    }
    for (int64_t at = 0; e == cudaSuccess && clip && at < std::max<int64_t>(count, 1); at += kMaxTable)
        e = any_pass(ts + at, std::min<int64_t>(kMaxTable, count - at), true, most, partial, n, max_norm,
                     at == 0 ? norm : nullptr, stream);
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

norm_status grad_workspace_bytes(int64_t count, int num_sms, size_t* bytes) {
    if (!bytes || count < 0 || num_sms < 1) return NORM_ERR_ARG;
    *bytes = static_cast<size_t>(libnorm::launches_of(count)) * static_cast<size_t>(num_sms) * libnorm::kCtasPerSm * 8;
    return NORM_OK;
}

}  // extern "C"
