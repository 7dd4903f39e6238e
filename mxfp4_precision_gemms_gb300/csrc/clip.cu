// clip.cu -- global gradient norm over many tensors, and clipping.
//
//   n = sqrt(sum over tensors and elements of g^2),  c = min(1, max_norm / (n + 1e-6)),  out = c * g
//
// Two launches.  The table of tensors travels in the kernels' parameters, so nothing is
// copied to the device and a captured graph replays it.  The tensors are cut into chunks of
// equal bytes.
//   1. Persistent CTAs sum the squares of their chunks in fp32 -- a thread's elements of one chunk, its
//      chunks, then trees over threads and CTAs, so that no chain of additions is long -- and
//      write one partial sum each.  (fp64 sums cost 20 us a call: every CTA of the second pass took
//      part in them, at 2 fp64 operations per SM and cycle.)
//   2. Each CTA adds the partial sums up in the same order, so that all have the same norm with
//      no atomics and no counter to reset, then scales its chunks, last read first: what the 129 MB
//      L2 still holds from the first pass is read from there.  Gradients that are clipped in
//      place by c == 1 are left as they are.
// HBM bandwidth bounds both passes of long calls, the two launches short ones.  A tensor that starts off 16 bytes is
// moved one element at a time: views into a flat buffer at an odd element, 872 MB of fp32 in 1165 us instead
// of 408 out of place, 252 instead of 130 where they are within the limit.
// Out of place, the second pass has a CTA for each chunk: CTAs that take one and end keep the accesses in
// address order (872 MB: 248 us against 272 for persistent ones and 257 for cudaMemcpy), and each
// loads its chunk before it adds up the norm.  In place it is persistent and looks at the norm
// first, because the ordinary step ends there: 5700 CTAs would take 15 us to find that out.
#include <algorithm>

#include "element.cuh"
#include "step_ops.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kClipThreads = 256;
constexpr int kClipCtasPerSm = 4;
constexpr int kMaxParts = 2048;  // partial sums of one call's launches together
constexpr int kBatch = 8;        // 16-byte units that a thread loads before it uses them
constexpr int kMinChunk = 12, kMaxChunk = 15;  // log2 of a chunk's bytes: one unit a thread .. kBatch
static_assert((1 << kMinChunk) == 16 * kClipThreads && (1 << kMaxChunk) == 16 * kClipThreads * kBatch, "units");

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
    int32_t chunk_log2;  // of its bytes
    int32_t in_place;  // every tensor is
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


// Chunk `chunk` of a launch: its tensor and the bytes of it.  The sums look at the gradient's alignment alone:
// where its clipped values go must not change the order of a sum, and so the norm.
struct Chunk {
    const uint8_t* in;
    uint8_t* out;
    int32_t bytes;
    bool is_bf16, vec;  // vec: 16-byte aligned
};
template <bool WRITES, int N>
__device__ __forceinline__ Chunk chunk_at(const ClipTable<N>& t, uint32_t chunk) {
    const int i = find_tensor(t, chunk);
    Chunk c;
    c.is_bf16 = t.is_bf16[i];
    const int64_t at = (int64_t)(chunk - t.first[i]) << t.chunk_log2;
    c.in = static_cast<const uint8_t*>(t.in[i]) + at;
    c.out = static_cast<uint8_t*>(t.out[i]) + at;
    c.bytes = (int32_t)min(int64_t(1) << t.chunk_log2, t.numel[i] * (c.is_bf16 ? 2 : 4) - at);
    c.vec = ((reinterpret_cast<uintptr_t>(c.in) | (WRITES ? reinterpret_cast<uintptr_t>(c.out) : 0)) & 15u) == 0;
    return c;
}

// This thread's units of a chunk (at most kBatch).
__device__ __forceinline__ void load_units(const Chunk& c, uint4 (&r)[kBatch]) {
    const int units = c.vec ? c.bytes / 16 : 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int u = threadIdx.x + k * kClipThreads;
        if (u < units) r[k] = reinterpret_cast<const uint4*>(c.in)[u];
    }
}

// f(element pointer index) over the elements that load_units leaves out.
template <class F>
__device__ __forceinline__ void for_rest(const Chunk& c, F&& f) {
    const int esz = c.is_bf16 ? 2 : 4;
    const int n = c.bytes / esz, first = c.vec ? c.bytes / 16 * (16 / esz) : 0;
    for (int i = first + threadIdx.x; i < n; i += kClipThreads) f(i);
}

__device__ __forceinline__ float chunk_squares(const Chunk& c) {
    uint4 r[kBatch];
    load_units(c, r);
    const int units = c.vec ? c.bytes / 16 : 0;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        if (threadIdx.x + k * kClipThreads >= units) break;
        const uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (c.is_bf16) {
                const float a = bf16_lo(w[j]), b = bf16_hi(w[j]);
                s0 = fmaf(a, a, s0);
                s1 = fmaf(b, b, s1);
            } else {
                const float a = __uint_as_float(w[j]);
                if (j & 1)
                    s1 = fmaf(a, a, s1);
                else
                    s0 = fmaf(a, a, s0);
            }
        }
    }
    for_rest(c, [&](int i) {
        const float v = c.is_bf16 ? load1(reinterpret_cast<const bf16*>(c.in) + i)
                                  : load1(reinterpret_cast<const float*>(c.in) + i);
        s0 = fmaf(v, v, s0);
    });
    return s0 + s1;
}

// The chunk's units (loaded before) and its other elements, times x.
__device__ __forceinline__ void chunk_scale(const Chunk& c, const uint4 (&r)[kBatch], float x) {
    const int units = c.vec ? c.bytes / 16 : 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int u = threadIdx.x + k * kClipThreads;
        if (u >= units) break;
        uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = c.is_bf16 ? pack_bf16(bf16_lo(w[j]) * x, bf16_hi(w[j]) * x)
                             : __float_as_uint(__uint_as_float(w[j]) * x);
        reinterpret_cast<uint4*>(c.out)[u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for_rest(c, [&](int i) {
        if (c.is_bf16) {
            const bf16* p = reinterpret_cast<const bf16*>(c.in) + i;
            store1(reinterpret_cast<bf16*>(c.out) + i, load1(p) * x);
        } else {
            const float* p = reinterpret_cast<const float*>(c.in) + i;
            store1(reinterpret_cast<float*>(c.out) + i, load1(p) * x);
        }
    });
}

// Sum over the CTA, the same value in every thread.
__device__ __forceinline__ float cta_sum(float v) {
    __shared__ float warp_sum[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum[threadIdx.x & (kClipThreads / 32 - 1)];
#pragma unroll
    for (int o = kClipThreads / 64; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// HBM-bound: 872 MB of fp32 gradients in 124 us (7.0 TB/s), 1.74 GB of bf16 ones in 241.
template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtasPerSm)
    squares_kernel(const __grid_constant__ ClipTable<N> t, float* part) {
    grid_dependency_wait();
    allow_dependent_launch();
    float sum = 0.f;
    const uint32_t chunks = t.first[t.n];
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) sum += chunk_squares(chunk_at<false>(t, c));
    sum = cta_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// HBM-bound: 872 MB into other buffers in 245 us (7.1 TB/s); 5 us where there is nothing to do.
template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtasPerSm)
    scale_kernel(const __grid_constant__ ClipTable<N> t, const float* part, int parts, float max_norm, float* norm) {
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t chunks = t.first[t.n];
    // This CTA's chunks from the last one down; the first of them is loaded beside the partial
    // sums, unless an in-place call may have nothing to do.
    int64_t ch = (int64_t)chunks - 1 - blockIdx.x;
    Chunk c;
    uint4 r[kBatch];
    if (ch >= 0) {
        c = chunk_at<true>(t, (uint32_t)ch);
        if (!t.in_place) load_units(c, r);
    }
    // The norm from the partial sums, the same in every CTA.
    float sum = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < parts; i += kClipThreads) sum += __ldcg(part + i);
    const float n = sqrtf(cta_sum(sum));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    const float q = max_norm / (n + 1e-6f);
    const float x = q > 1.f ? 1.f : q;  // NaN stays NaN
    if (ch < 0 || (x == 1.f && t.in_place)) return;
    if (t.in_place) load_units(c, r);
    for (;;) {
        if (x != 1.f || c.in != c.out) chunk_scale(c, r, x);
        ch -= gridDim.x;
        if (ch < 0) return;
        c = chunk_at<true>(t, (uint32_t)ch);
        load_units(c, r);
    }
}

template <int N>
void fill_table(ClipTable<N>& t, const mxfp4_grad* g, int n, int chunk_log2) {
    t.n = n;
    t.chunk_log2 = chunk_log2;
    t.in_place = 1;
    uint32_t chunk = 0;
    for (int i = 0; i < n; ++i) {
        t.in[i] = g[i].grad;
        t.out[i] = g[i].out;
        t.numel[i] = g[i].numel;
        if (g[i].grad != g[i].out) t.in_place = 0;
        t.is_bf16[i] = g[i].dtype == MXFP4_OUT_BF16;
        t.first[i] = chunk;
        const int64_t bytes = g[i].numel * (t.is_bf16[i] ? 2 : 4);
        chunk += (uint32_t)((bytes + (int64_t(1) << chunk_log2) - 1) >> chunk_log2);
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
cudaError_t launch_clip(const mxfp4_grad* g, int n, int chunk_log2, int ctas, float max_norm, float* norm, float* part,
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
        const uint32_t chunks = t.first[t.n];
        const uint32_t grid = std::max<uint32_t>(1u, t.in_place ? std::min<uint32_t>((uint32_t)ctas, chunks) : chunks);
        cudaError_t e = launch_overlapped(scale_kernel<N>, dim3(grid), dim3(kClipThreads), 0, s, 1, true, t,
                                          const_cast<const float*>(part), parts, max_norm, norm);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

constexpr int64_t kMaxElements = int64_t(1) << 42;  // chunks stay within 31 bits
constexpr int kMaxGrads = 1 << 20;  // 1024 tables: still two partial sums each

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mxfp4_clip_grad_norm_workspace_bytes(int n) {
    return n < 0 || n > kMaxGrads ? 0 : kMaxParts * sizeof(float);
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
        if (g.numel > kMaxElements || total > kMaxElements)
            return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: more than 2^42 elements", what);
        total += g.numel;
    }
    if (!ws || ws_bytes < kMaxParts * sizeof(float))
        return record_error(MXFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", what, kMaxParts * sizeof(float));
    if (reinterpret_cast<uintptr_t>(ws) % 256)
        return record_error(MXFP4_ERR_MISALIGNED, "%s: workspace not 256-byte aligned", what);
    mxfp4_status st = ensure_device();
    if (st) return st;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    const int ctas = std::min(kMaxParts, sms * kClipCtasPerSm);
    // Chunks of kBatch units a thread where there is work enough, shorter ones where that spreads a
    // short call over more CTAs.
    int chunk_log2 = kMinChunk;
    while (chunk_log2 < kMaxChunk && (total * 4 >> chunk_log2) > 2 * ctas) ++chunk_log2;
    float* part = static_cast<float*>(ws);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    e = n <= kSmallTable ? launch_clip<kSmallTable>(grads, n, chunk_log2, ctas, max_norm, norm, part, s)
                         : launch_clip<kLargeTable>(grads, n, chunk_log2, ctas, max_norm, norm, part, s);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}
