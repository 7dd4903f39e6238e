// clip.cu -- global gradient norm over many tensors, and clipping.
//
//   n = sqrt(sum over tensors and elements of g^2),  c = min(1, max_norm / (n + 1e-6)),  out = c * g
//
// Two launches.  The table of tensors travels in the kernels' parameters, so nothing is
// copied to the device and a captured graph replays it.  The tensors are cut into chunks of
// equal size that the CTAs take in turn.
//   1. Each CTA sums the squares of its chunks -- fp32 over a thread's elements of one chunk, fp64
//      from there on -- and writes one partial sum.
//   2. Each CTA adds the partial sums up in the same order, so that all have the same norm with
//      no atomics and no counter to reset, then scales its chunks, last read first: what the 129 MB
//      L2 still holds from the first pass is read from there.  A gradient that is clipped in
//      place by c == 1 is left as it is.
// HBM bandwidth bounds both passes of long calls, the two launches short ones.
#include <algorithm>

#include "element.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kClipThreads = 256;
constexpr int kClipCtasPerSm = 8;
constexpr int kMaxParts = 2048;  // partial sums of one call's launches together
constexpr int64_t kMaxChunk = 16384, kMinChunk = 2048;  // elements of a chunk (a power of two)

// Up to N tensors of one launch; chunk c of the launch belongs to the tensor i with
// first[i] <= c < first[i + 1].
template <int N>
struct ClipTable {
    const void* in[N];
    void* out[N];
    int64_t numel[N];
    uint32_t first[N + 1];
    uint8_t is_bf16[N];
    int32_t n;
    int32_t chunk_log2;
};
// Kernel parameters hold 32764 bytes.  The small table is for the usual few tensors: a launch
// copies its parameters, all of them.
constexpr int kSmallTable = 64, kLargeTable = 1024;
static_assert(sizeof(ClipTable<kLargeTable>) + 64 <= 32764, "kernel parameters");

template <int N>
__device__ __forceinline__ int find_tensor(const ClipTable<N>& t, uint32_t chunk) {
    int lo = 0, hi = t.n;  // first[lo] <= chunk < first[hi]; empty tensors have no chunk
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}


// Sum of squares of n elements at p over the CTA's threads (this thread's share).
template <class T>
__device__ __forceinline__ float chunk_squares(const T* p, int64_t n) {
    float s0 = 0.f, s1 = 0.f;
    int64_t done = 0;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const int64_t units = n / 8;
#pragma unroll 4
        for (int64_t u = threadIdx.x; u < units; u += kClipThreads) {
            float v[8];
            unpack8(load8(p + u * 8), v);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                s0 = fmaf(v[j], v[j], s0);
                s1 = fmaf(v[j + 1], v[j + 1], s1);
            }
        }
        done = units * 8;
    }
#pragma unroll 4
    for (int64_t i = done + threadIdx.x; i < n; i += kClipThreads) {
        const float v = load1(p + i);
        s0 = fmaf(v, v, s0);
    }
    return s0 + s1;
}

template <class T>
__device__ __forceinline__ void chunk_scale(const T* p, T* q, int64_t n, float c) {
    int64_t done = 0;
    if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0) {
        const int64_t units = n / 8;
#pragma unroll 4
        for (int64_t u = threadIdx.x; u < units; u += kClipThreads) {
            float v[8];
            unpack8(load8(p + u * 8), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= c;
            store8(q + u * 8, v);
        }
        done = units * 8;
    }
#pragma unroll 4
    for (int64_t i = done + threadIdx.x; i < n; i += kClipThreads) store1(q + i, load1(p + i) * c);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtasPerSm)
    squares_kernel(const __grid_constant__ ClipTable<N> t, double* part) {
    __shared__ double warp_sum[kClipThreads / 32];
    grid_dependency_wait();
    double sum = 0.0;
    const uint32_t chunks = t.first[t.n];
    const int64_t len = int64_t(1) << t.chunk_log2;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = find_tensor(t, c);
        const int64_t at = (int64_t)(c - t.first[i]) << t.chunk_log2;
        const int64_t n = min(len, t.numel[i] - at);
        sum += t.is_bf16[i] ? chunk_squares(static_cast<const bf16*>(t.in[i]) + at, n)
                            : chunk_squares(static_cast<const float*>(t.in[i]) + at, n);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int w = 0; w < kClipThreads / 32; ++w) all += warp_sum[w];
        part[blockIdx.x] = all;
    }
}

// The norm from the partial sums, the same in every CTA.
__device__ __forceinline__ float norm_of(const double* part, int parts) {
    __shared__ double warp_sum[kClipThreads / 32];
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipThreads) sum += __ldcg(part + i);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < kClipThreads / 32; ++w) all += warp_sum[w];
    return (float)sqrt(all);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtasPerSm)
    scale_kernel(const __grid_constant__ ClipTable<N> t, const double* part, int parts, float max_norm, float* norm) {
    grid_dependency_wait();
    const float n = norm_of(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    const float r = max_norm / (n + 1e-6f);
    const float c = r > 1.f ? 1.f : r;  // NaN stays NaN
    const uint32_t chunks = t.first[t.n];
    const int64_t len = int64_t(1) << t.chunk_log2;
    if (blockIdx.x >= chunks) return;
    const uint32_t turns = (chunks - 1 - blockIdx.x) / gridDim.x;
    for (int64_t k = turns; k >= 0; --k) {
        const uint32_t ch = blockIdx.x + (uint32_t)k * gridDim.x;
        const int i = find_tensor(t, ch);
        if (c == 1.f && t.in[i] == t.out[i]) continue;
        const int64_t at = (int64_t)(ch - t.first[i]) << t.chunk_log2;
        const int64_t m = min(len, t.numel[i] - at);
        if (t.is_bf16[i])
            chunk_scale(static_cast<const bf16*>(t.in[i]) + at, static_cast<bf16*>(t.out[i]) + at, m, c);
        else
            chunk_scale(static_cast<const float*>(t.in[i]) + at, static_cast<float*>(t.out[i]) + at, m, c);
    }
}

template <int N>
void fill_table(ClipTable<N>& t, const mxfp4_grad* g, int n, int chunk_log2) {
    t.n = n;
    t.chunk_log2 = chunk_log2;
    uint32_t chunk = 0;
    for (int i = 0; i < n; ++i) {
        t.in[i] = g[i].grad;
        t.out[i] = g[i].out;
        t.numel[i] = g[i].numel;
        t.is_bf16[i] = g[i].dtype == MXFP4_OUT_BF16;
        t.first[i] = chunk;
        chunk += (uint32_t)((g[i].numel + (int64_t(1) << chunk_log2) - 1) >> chunk_log2);
    }
    t.first[n] = chunk;
}

cudaError_t sm_count(int* sms) {
    static DeviceSlots slots;
    return per_device_setting(slots, sms, [&](int dev, int* n) {
        return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
    });
}

// Launches both passes over tables of N tensors each (several where n > N).
template <int N>
cudaError_t launch_clip(const mxfp4_grad* g, int n, int chunk_log2, int ctas, float max_norm, float* norm, double* part,
                        cudaStream_t s) {
    const int tables = n > N ? (n + N - 1) / N : 1;
    const int most = std::min(ctas, kMaxParts / tables);
    ClipTable<N> t;
    int parts = 0;
    for (int k = 0; k < tables; ++k) {
        fill_table(t, g + k * N, std::min(N, n - k * N), chunk_log2);
        const int grid = (int)std::max<uint32_t>(1u, std::min<uint32_t>((uint32_t)most, t.first[t.n]));
        cudaError_t e = launch_overlapped(squares_kernel<N>, dim3(grid), dim3(kClipThreads), 0, s, 1, true, t, part + parts);
        if (e != cudaSuccess) return e;
        parts += grid;
    }
    for (int k = tables - 1; k >= 0; --k) {  // last read first
        if (tables > 1) fill_table(t, g + k * N, std::min(N, n - k * N), chunk_log2);
        const int grid = (int)std::max<uint32_t>(1u, std::min<uint32_t>((uint32_t)ctas, t.first[t.n]));
        cudaError_t e = launch_overlapped(scale_kernel<N>, dim3(grid), dim3(kClipThreads), 0, s, 1, true, t,
                                          const_cast<const double*>(part), parts, max_norm, norm);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

constexpr int kMaxGrads = 1 << 20;  // 1024 tables: still two partial sums each

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mxfp4_clip_grad_norm_workspace_bytes(int n) {
    return n < 0 || n > kMaxGrads ? 0 : kMaxParts * sizeof(double);
}

extern "C" mxfp4_status mxfp4_clip_grad_norm(const mxfp4_grad* grads, int n, float max_norm, float* norm, void* ws,
                                             size_t ws_bytes, mxfp4_stream_t stream) {
    const char* what = "clip_grad_norm";
    if (n < 0) return record_error(MXFP4_ERR_INVALID_ARG, "%s: negative count", what);
    if (n > kMaxGrads) return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: more than %d gradients", what, kMaxGrads);
    if (n > 0 && !grads) return record_error(MXFP4_ERR_INVALID_ARG, "%s: grads is NULL", what);
    if (!(max_norm >= 0.f)) return record_error(MXFP4_ERR_INVALID_ARG, "%s: max_norm must be >= 0", what);
    if (!norm) return record_error(MXFP4_ERR_INVALID_ARG, "%s: norm is NULL", what);
    if (reinterpret_cast<uintptr_t>(norm) % 4) return record_error(MXFP4_ERR_MISALIGNED, "%s: norm misaligned", what);
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        const mxfp4_grad& g = grads[i];
        if (g.dtype != MXFP4_OUT_F32 && g.dtype != MXFP4_OUT_BF16)
            return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad dtype %d of gradient %d", what, g.dtype, i);
        if (g.reserved != 0) return record_error(MXFP4_ERR_INVALID_ARG, "%s: reserved must be 0", what);
        if (g.numel < 0) return record_error(MXFP4_ERR_INVALID_ARG, "%s: negative size of gradient %d", what, i);
        if (g.numel == 0) continue;
        if (!g.grad || !g.out) return record_error(MXFP4_ERR_INVALID_ARG, "%s: gradient %d has a NULL pointer", what, i);
        const uintptr_t esz = g.dtype == MXFP4_OUT_BF16 ? 2 : 4;
        if (reinterpret_cast<uintptr_t>(g.grad) % esz || reinterpret_cast<uintptr_t>(g.out) % esz)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: gradient %d not aligned to its type", what, i);
        if (g.numel > (int64_t(1) << 44) || total > (int64_t(1) << 44))
            return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: more than 2^44 elements", what);
        total += g.numel;
    }
    if (!ws || ws_bytes < kMaxParts * sizeof(double))
        return record_error(MXFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", what, kMaxParts * sizeof(double));
    if (reinterpret_cast<uintptr_t>(ws) % 256)
        return record_error(MXFP4_ERR_MISALIGNED, "%s: workspace not 256-byte aligned", what);
    mxfp4_status st = ensure_device();
    if (st) return st;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    const int ctas = std::min(kMaxParts, sms * kClipCtasPerSm);
    // Chunks of kMaxChunk elements where there is enough work, shorter ones (down to one vector
    // a thread) where that spreads a short call over more CTAs, longer ones past 2^45 elements
    // in sight of the 32-bit chunk index.
    int chunk_log2 = 11;
    while ((int64_t(1) << chunk_log2) < kMaxChunk && (total >> chunk_log2) > 2 * ctas) ++chunk_log2;
    while ((total >> chunk_log2) > (int64_t(1) << 30)) ++chunk_log2;
    static_assert(kMinChunk == 1 << 11 && kMinChunk == 8 * kClipThreads, "one vector a thread");
    double* part = static_cast<double*>(ws);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    e = n <= kSmallTable ? launch_clip<kSmallTable>(grads, n, chunk_log2, ctas, max_norm, norm, part, s)
                         : launch_clip<kLargeTable>(grads, n, chunk_log2, ctas, max_norm, norm, part, s);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}
