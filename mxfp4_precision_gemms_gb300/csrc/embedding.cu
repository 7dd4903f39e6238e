// embedding.cu -- embedding lookup with scaling, and the table's gradient by sorted tokens.
//
//   y[t, :]  = s * w[id_t, :]
//   dw[v, :] (+)= s * sum over { t : id_t = v } of dy[t, :]      (fp32, t in a fixed order)
//
// Both only move data: the lookup reads and writes tokens x dim elements, the gradient reads
// them once and writes the table (or reads and writes the rows that occur, when it adds to
// the table).  HBM bandwidth bounds every long call, launch latency the short ones.
//
// The gradient is three launches.
//   1. Sort.  One CTA, or a cluster of up to eight, sorts (id, token) pairs by id, stably, with a
//      least-significant-digit radix sort of 9 bits a pass (two passes up to 262143 ids): each
//      warp owns a contiguous run of tokens and counts its digits with match.any, so that the
//      order within a digit is the order of the tokens.  The other CTAs of the launch meanwhile
//      clear the table.
//   2. Sum.  The sorted tokens are cut into chunks of kChunk.  A CTA owns one chunk and one slab
//      of columns and adds its rows up in registers; a row of the table whose tokens all lie in
//      the chunk is finished there.  A run that crosses a chunk's border leaves an fp32 partial
//      sum, so a very frequent token is shared out over many CTAs.
//   3. Join.  The partial sums of each crossing run are added in chunk order.
// A few tokens are not sorted: one CTA for each token and slab of columns looks its id up among the
// others and, where it is the first of its id, adds up their rows.
// Which additions are made in which order depends on the ids alone, never on timing.
#include <algorithm>

#include "element.cuh"
#include "step_ops.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

// ---------------------------------------------------------------- lookup
constexpr int kLookupThreads = 256;
constexpr int kLookupUnits = 4;  // units (8 elements, or one) in flight per lane

// One warp per row segment of 32 * kLookupUnits units, its loads in flight together.  8192 rows of 8 KB take
// 17 us a call (134 MB; HBM alone 20 us, part of the rows stays in L2), one row 2 us.
template <class W, class Y, bool VEC>
__global__ void __launch_bounds__(kLookupThreads)
    lookup_kernel(const void* ids, int is64, int64_t tokens, const W* w, int64_t vocab, int64_t dim, int64_t ldw,
                  float scale, Y* y, int64_t ldy, uint32_t segs, uint32_t* status) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t wid = (int64_t)blockIdx.x * (kLookupThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = wid / segs;
    if (t >= tokens) return;
    const int64_t seg = wid - t * segs;
    const int64_t id = load_id(ids, is64, t);
    const bool good = id >= 0 && id < vocab;
    if (!good && seg == 0 && lane == 0) atomicOr(status, kStatusBadIndex);
    const W* src = w + (good ? id : 0) * ldw;
    Y* dst = y + t * ldy;
    constexpr int U = VEC ? 8 : 1;
    const int64_t units = VEC ? dim / 8 : dim;
    const int64_t u0 = seg * (32 * kLookupUnits) + lane;
    if constexpr (VEC) {
        Raw8<W> r[kLookupUnits];
#pragma unroll
        for (int i = 0; i < kLookupUnits; ++i)
            if (good && u0 + i * 32 < units) r[i] = load8(src + (u0 + i * 32) * U);
#pragma unroll
        for (int i = 0; i < kLookupUnits; ++i) {
            if (u0 + i * 32 >= units) break;
            float v[8] = {};
            if (good) {
                unpack8(r[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= scale;
            }
            store8(dst + (u0 + i * 32) * U, v);
        }
    } else {
        float v[kLookupUnits];
#pragma unroll
        for (int i = 0; i < kLookupUnits; ++i) v[i] = good && u0 + i * 32 < units ? load1(src + u0 + i * 32) : 0.f;
#pragma unroll
        for (int i = 0; i < kLookupUnits; ++i)
            if (u0 + i * 32 < units) store1(dst + u0 + i * 32, good ? v[i] * scale : 0.f);
    }
}

// ---------------------------------------------------------------- sort (and clear)
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtasMost = 8;  // the portable cluster size
constexpr uint32_t kSortTokens = 2048;  // tokens for each CTA: more CTAs pay for their barriers above that
constexpr int kBits = 9;
constexpr int kBins = 1 << kBits;
// counters [warp][bin], this CTA's bin totals, the cluster-wide offsets, scan scratch
constexpr int kSortSmem = (kSortWarps * kBins + 2 * kBins + 32) * 4;
// Bytes that a clearing CTA clears, two 16-byte stores a thread.  CTAs that each clear one stretch and
// end keep the stores in address order: 7.65 TB/s over a 1.05 GB table, where persistent CTAs
// reached 6.4 with plain stores and 6.3 to 6.9 with bulk copies of a zeroed buffer.
constexpr int64_t kClearBytes = 2 * 16 * kSortThreads;
constexpr int kSortItems = 4;  // tokens of a lane that are loaded together
constexpr int kChunk = 32;     // sorted tokens of a chunk
constexpr uint32_t kLongRun = 16;  // chunks

// A run of one id that crosses a chunk's border: its first chunk, and the one behind its last.
struct Run {
    uint32_t key, first, end;
};

struct SortParams {
    const void* ids;
    int32_t is64;
    int32_t passes;
    uint32_t tokens;
    int64_t vocab, padding_id;
    uint2* buf[2];  // (key, token); the last pass writes buf[0]
    uint32_t* num_runs;  // [2]: cleared here, counted by the sums
    uint32_t* status;
    // clearing: rows of row_bytes, pitch_bytes apart
    uint8_t* dw;
    int64_t rows, row_bytes, pitch_bytes;
    int32_t clear;
    int32_t clear_flat;  // contiguous and 16-byte aligned: one run of bytes
    int32_t clear_vec;   // 16-byte aligned rows of a multiple of 16 bytes
};

// Whether a token's row belongs to the gradient; one outside the vocabulary is reported.
__device__ __forceinline__ bool takes_part(int64_t id, int64_t vocab, int64_t padding_id, uint32_t* status) {
    if (id >= 0 && id == padding_id) return false;
    if (id >= 0 && id < vocab) return true;
    atomicOr(status, kStatusBadIndex);
    return false;
}

// kSortItems (key, token) pairs of a lane, its tokens 32 apart from t0 on: in the first pass the key is
// the token's id, or `vocab` (behind every row) when it is left out.
__device__ __forceinline__ void load_pairs(const SortParams& p, const uint2* in, bool first_pass, uint32_t t0,
                                           uint32_t end, uint2 (&kv)[kSortItems]) {
    if (!first_pass) {
#pragma unroll
        for (int k = 0; k < kSortItems; ++k) {
            const uint32_t t = t0 + k * 32;
            kv[k] = t < end ? __ldcg(&in[t]) : make_uint2(0u, 0u);
        }
        return;
    }
    int64_t id[kSortItems];  // all loads before the first use
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
        const uint32_t t = t0 + k * 32;
        id[k] = t < end ? load_id(p.ids, p.is64, t) : 0;
    }
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
        const uint32_t t = t0 + k * 32;
        const bool on = t < end && takes_part(id[k], p.vocab, p.padding_id, p.status);
        kv[k] = make_uint2((uint32_t)(on ? id[k] : p.vocab), t);
    }
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Barrier over the sorting CTAs, with their global writes visible to all of them.
template <int CTAS>
__device__ __forceinline__ void sort_sync() {
    if constexpr (CTAS > 1)
        cluster_sync();
    else
        __syncthreads();
}

// Latency-bound: 14 us for 8192 tokens, 22 us for 32768, most of it barriers and trips to L2 and back.  Nine bits a
// pass are two passes for the usual vocabularies; wider digits would not fit their counters.
template <int CTAS>
__device__ void sort_tokens(const SortParams& p, uint32_t* smem) {
    if (p.tokens == 0) return;  // nothing to sort, and no workspace: the launch only clears
    uint32_t* count = smem;                       // [kSortWarps][kBins]
    uint32_t* total = count + kSortWarps * kBins;  // [kBins]
    uint32_t* base = total + kBins;                // [kBins]
    uint32_t* wsum = base + kBins;                 // [32]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = CTAS > 1 ? cluster_ctarank() : 0;
    // contiguous run of tokens of this warp, a multiple of 32 long
    const uint32_t per_warp = ((p.tokens + CTAS * kSortWarps * 32 - 1) / (CTAS * kSortWarps * 32)) * 32;
    const uint64_t first = (uint64_t)(rank * kSortWarps + warp) * per_warp;
    const uint32_t begin = (uint32_t)(first < p.tokens ? first : p.tokens);
    const uint32_t end = (uint32_t)(first + per_warp < p.tokens ? first + per_warp : p.tokens);
    // warps of this CTA that have tokens
    const uint64_t mine_from = (uint64_t)rank * kSortWarps * per_warp;
    const uint32_t warps = mine_from >= p.tokens ? 0u
                                                  : (uint32_t)min((uint64_t)kSortWarps,
                                                                  (p.tokens - mine_from + per_warp - 1) / per_warp);
    uint32_t* mine = count + warp * kBins;
    if (rank == 0 && tid < 2) p.num_runs[tid] = 0;

    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * kBits;
        const uint2* in = p.buf[(p.passes - pass) & 1];
        uint2* out = p.buf[(p.passes - pass - 1) & 1];
        for (uint32_t i = tid; i < warps * (kBins / 4); i += kSortThreads)
            reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        for (uint32_t t0 = begin; t0 < end; t0 += 32 * kSortItems) {
            uint2 kv[kSortItems];
            load_pairs(p, in, pass == 0, t0 + lane, end, kv);
#pragma unroll
            for (int k = 0; k < kSortItems; ++k) {
                const bool on = t0 + k * 32 + lane < end;
                const uint32_t mask = __ballot_sync(0xffffffffu, on);
                if (on) {
                    const uint32_t d = (kv[k].x >> shift) & (kBins - 1);
                    const uint32_t peers = __match_any_sync(mask, d);
                    if ((peers & ((1u << lane) - 1)) == 0) mine[d] += __popc(peers);
                }
                __syncwarp();
            }
        }
        __syncthreads();
        uint32_t before = 0, all = 0;
        if (tid < kBins) {  // exclusive over the warps of this CTA
            uint32_t run = 0;
            for (uint32_t w0 = 0; w0 < warps; w0 += 8) {
                uint32_t c[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] = w0 + j < warps ? count[(w0 + j) * kBins + tid] : 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (w0 + j < warps) count[(w0 + j) * kBins + tid] = run;
                    run += c[j];
                }
            }
            total[tid] = run;
            all = run;
        }
        if constexpr (CTAS > 1) {  // the other CTAs' totals
            cluster_sync();
            if (tid < kBins) {
                const uint32_t a = smem_u32(total + tid);
                uint32_t c[CTAS];
#pragma unroll
                for (int r = 0; r < CTAS; ++r) c[r] = ld_cluster_u32(mapa_shared(a, r));
                all = 0;
#pragma unroll
                for (int r = 0; r < CTAS; ++r) {
                    before += r < (int)rank ? c[r] : 0u;
                    all += c[r];
                }
            }
        }
        // exclusive scan of `all` over the bins (16 warps of 32 bins)
        uint32_t inc = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += n;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        if (tid < kBins) {
            uint32_t lower = lane < warp ? wsum[lane] : 0u;  // warp < 16
            lower = __reduce_add_sync(0xffffffffu, lower);
            base[tid] = lower + inc - all + before;
        }
        __syncthreads();
        for (uint32_t t0 = begin; t0 < end; t0 += 32 * kSortItems) {
            uint2 kv[kSortItems];
            load_pairs(p, in, pass == 0, t0 + lane, end, kv);
#pragma unroll
            for (int k = 0; k < kSortItems; ++k) {
                const bool on = t0 + k * 32 + lane < end;
                const uint32_t mask = __ballot_sync(0xffffffffu, on);
                uint32_t d = 0, peers = 0;
                if (on) {
                    d = (kv[k].x >> shift) & (kBins - 1);
                    peers = __match_any_sync(mask, d);
                    out[base[d] + mine[d] + __popc(peers & ((1u << lane) - 1))] = kv[k];
                }
                __syncwarp();
                if (on && (peers & ((1u << lane) - 1)) == 0) mine[d] += __popc(peers);
                __syncwarp();
            }
        }
        // The pass's output is visible to all of them, and no CTA's totals are still being read,
        // before the next pass starts.
        sort_sync<CTAS>();
    }
}

// Zeroes the table's part of CTA `part` of `parts`.
__device__ __forceinline__ void clear_table(const SortParams& p, uint32_t part, uint32_t parts) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (p.clear_flat) {  // one run of bytes, kClearBytes of it here
        const int64_t all = p.rows * p.row_bytes;
        const int64_t at = part * kClearBytes + threadIdx.x * 16;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t o = at + k * 16 * kSortThreads;
            if (o + 16 <= all)
                *reinterpret_cast<uint4*>(p.dw + o) = zero;
            else  // the last bytes of a table that does not fill 16; every element is a multiple of two
                for (int64_t b = o; b < all; b += 2) *reinterpret_cast<uint16_t*>(p.dw + b) = 0;
        }
        return;
    }
    for (int64_t r = part; r < p.rows; r += parts) {
        uint8_t* row = p.dw + r * p.pitch_bytes;
        if (p.clear_vec)
            for (int64_t i = threadIdx.x; i < p.row_bytes / 16; i += kSortThreads) reinterpret_cast<uint4*>(row)[i] = zero;
        else
            for (int64_t i = threadIdx.x; i < p.row_bytes / 2; i += kSortThreads) reinterpret_cast<uint16_t*>(row)[i] = 0;
    }
}

template <int CTAS>
__global__ void __launch_bounds__(kSortThreads, 2) sort_clear_kernel(const __grid_constant__ SortParams p) {
    extern __shared__ __align__(16) uint32_t smem[];
    grid_dependency_wait();
    allow_dependent_launch();
    if (blockIdx.x < CTAS)
        sort_tokens<CTAS>(p, smem);
    else
        clear_table(p, blockIdx.x - CTAS, gridDim.x - CTAS);
}

// ---------------------------------------------------------------- sum and join
// Rows loaded before they are added; with the rows of dw that they are added to, half as many leave
// registers for six CTAs an SM (32768 tokens into 32000 x 4096 fp32: 136 us with 8, 125 with 4, 127 with 2).
constexpr int kAhead = 8, kAheadAcc = 4;
constexpr int kSumThreads = 128;

struct SumParams {
    const uint2* sorted;
    uint32_t tokens;
    int64_t vocab, dim, lddy, lddw;
    float scale;
    int32_t accumulate;
    float* part;  // [chunks][2][dim]: a run that came in from the left, a run that goes out to the right
    Run* runs;           // short runs from the front, long ones from the back; in no particular order
    uint32_t* num_runs;  // [2]: short, long
    uint32_t chunks;
};

// What a row of the table becomes: `old` is what it holds where the gradient is added to it.
__device__ __forceinline__ float finished(float sum, float old, const SumParams& p) {
    return p.accumulate ? fmaf(p.scale, sum, old) : p.scale * sum;
}

// Enters the run that starts in this chunk and goes on in the next into its list.
__device__ __forceinline__ void enter_run(const SumParams& p, uint32_t chunk, uint32_t key) {
    // The first key of chunk lo is `key`, that of chunk hi is not.  Most runs end soon: strides
    // that double first, then halving between the last two.
    uint32_t lo = chunk + 1, hi = p.chunks;
    for (uint32_t step = 1; lo + step < hi; step *= 2) {
        if (__ldcg(&p.sorted[(uint64_t)(lo + step) * kChunk]).x != key) {
            hi = lo + step;
            break;
        }
        lo += step;
    }
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (__ldcg(&p.sorted[(uint64_t)mid * kChunk]).x == key)
            lo = mid;
        else
            hi = mid;
    }
    const bool is_long = hi - chunk > kLongRun;
    const uint32_t at = atomicAdd(&p.num_runs[is_long ? 1 : 0], 1u);
    p.runs[is_long ? p.chunks - 1 - at : at] = {key, chunk, hi};
}

// One chunk of sorted tokens x one slab of columns (8 per thread, or one).  HBM-bound: 8192 rows of 8 KB
// in 17 us, 32768 of them added to fp32 rows in 91 (563 MB, 6.2 TB/s).  ACC: dw is added to;
// the rows that end in the chunk are loaded along with the tokens' rows.
template <class DY, class DW, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumParams p, const DY* dy, DW* dw) {
    constexpr int U = VEC ? 8 : 1;
    constexpr int AHEAD = ACC ? kAheadAcc : kAhead;
    __shared__ uint2 kv[kChunk + 2];  // with the neighbours' keys on both sides
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t slab = blockIdx.x / p.chunks, chunk = blockIdx.x - slab * p.chunks;
    const uint32_t begin = chunk * kChunk;
    const uint32_t n = min((uint32_t)kChunk, p.tokens - begin);
    for (int i = threadIdx.x; i < (int)n + 2; i += kSumThreads) {
        const int64_t at = (int64_t)begin + i - 1;
        kv[i] = at >= 0 && at < p.tokens ? p.sorted[at] : make_uint2(0xffffffffu, 0);
    }
    __syncthreads();
    const uint32_t none = (uint32_t)p.vocab;  // the key of tokens that are left out
    if (kv[1].x == none) return;
    if (slab == 0 && threadIdx.x == kSumThreads - 1) {
        const uint32_t key = kv[n].x;
        if (key != none && kv[n + 1].x == key && kv[0].x != key) enter_run(p, chunk, key);
    }
    const int64_t col = ((int64_t)slab * kSumThreads + threadIdx.x) * U;
    if (col >= p.dim) return;

    float acc[U] = {};
    for (uint32_t i0 = 0; i0 < n; i0 += AHEAD) {
        Raw8<DY> raw[VEC ? AHEAD : 1];
        Raw8<DW> old[VEC && ACC ? AHEAD : 1];
        float one[VEC ? 1 : AHEAD], old1[VEC ? 1 : AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const uint32_t i = i0 + a;
            if (i >= n || kv[1 + i].x == none) break;
            const uint32_t key = kv[1 + i].x;
            const DY* src = dy + (int64_t)kv[1 + i].y * p.lddy + col;
            if constexpr (VEC)
                raw[a] = load8(src);
            else
                one[a] = load1(src);
            if (ACC && kv[2 + i].x != key && kv[0].x != key) {
                if constexpr (VEC)
                    old[a] = load8(dw + (int64_t)key * p.lddw + col);
                else
                    old1[a] = load1(dw + (int64_t)key * p.lddw + col);
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const uint32_t i = i0 + a;
            if (i >= n || kv[1 + i].x == none) break;
            if constexpr (VEC) {
                float v[8];
                unpack8(raw[a], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += v[j];
            } else {
                acc[0] += one[a];
            }
            const uint32_t key = kv[1 + i].x;
            const bool last = kv[2 + i].x != key;
            if (!last && i + 1 < n) continue;  // the run goes on inside the chunk
            // The run ends here, or the chunk does.  It came in from the left if the chunk's
            // first key and the one before it are the same.
            const bool from_left = kv[0].x == key;
            if (last && !from_left) {
                DW* dst = dw + (int64_t)key * p.lddw + col;
                if constexpr (VEC) {
                    float v[8] = {};
                    if constexpr (ACC) unpack8(old[a], v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = finished(acc[j], v[j], p);
                    store8(dst, v);
                } else {
                    store1(dst, finished(acc[0], ACC ? old1[a] : 0.f, p));
                }
            } else {
                float* to = p.part + ((int64_t)chunk * 2 + (from_left ? 0 : 1)) * p.dim + col;
                if constexpr (VEC)
                    store8(to, acc);
                else
                    to[0] = acc[0];
            }
#pragma unroll
            for (int j = 0; j < U; ++j) acc[j] = 0.f;
        }
    }
}

// Joins the crossing runs, one run and one slab of 32 units at a time: a short run's chunks are
// added by one warp in turn, a long run's by the CTA's warps, each taking every eighth, and their
// sums in the warps' order.  5 us after 8192 tokens, 12 after 32768: a few dependent reads of L2.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

template <class DW, bool VEC>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const SumParams p, DW* dw, uint32_t slabs) {
    constexpr int U = VEC ? 4 : 1;
    __shared__ float part[kJoinWarps][32 * U];
    grid_dependency_wait();
    allow_dependent_launch();
    const uint64_t shorts = (uint64_t)p.num_runs[0] * slabs, longs = (uint64_t)p.num_runs[1] * slabs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // chunk c of a run: slot 1 (going out) where it starts, slot 0 (coming in) after that
    auto add = [&](float (&acc)[U], const Run& run, uint32_t c, int64_t col) {
        const float* src = p.part + ((int64_t)c * 2 + (c == run.first ? 1 : 0)) * p.dim + col;
        if constexpr (VEC) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
        } else {
            acc[0] += src[0];
        }
    };
    for (uint64_t item = blockIdx.x; item < longs; item += gridDim.x) {
        const uint32_t slab = (uint32_t)(item % slabs);
        const Run run = p.runs[p.chunks - 1 - item / slabs];
        const int64_t col0 = (int64_t)slab * 32 * U, col = col0 + lane * U;
        float acc[U] = {};
        if (col < p.dim) {
#pragma unroll 4
            for (uint32_t c = run.first + warp; c < run.end; c += kJoinWarps) add(acc, run, c, col);
        }
        __syncthreads();  // the item before has been read
#pragma unroll
        for (int j = 0; j < U; ++j) part[warp][lane * U + j] = acc[j];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * U; i += kJoinThreads) {
            if (col0 + i >= p.dim) break;
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k) sum += part[k][i];
            DW* dst = dw + (int64_t)run.key * p.lddw + col0 + i;
            store1(dst, finished(sum, p.accumulate ? load1(dst) : 0.f, p));
        }
    }
    for (uint64_t item = (uint64_t)blockIdx.x * kJoinWarps + warp; item < shorts; item += (uint64_t)gridDim.x * kJoinWarps) {
        const uint32_t slab = (uint32_t)(item % slabs);
        const Run run = p.runs[item / slabs];
        const int64_t col = ((int64_t)slab * 32 + lane) * U;
        if (col >= p.dim) continue;
        DW* dst = dw + (int64_t)run.key * p.lddw + col;
        float acc[U] = {}, old[U] = {};
        if (p.accumulate) {
            if constexpr (VEC)
                load4(dst, old);
            else
                old[0] = load1(dst);
        }
#pragma unroll 4
        for (uint32_t c = run.first; c < run.end; ++c) add(acc, run, c, col);
#pragma unroll
        for (int j = 0; j < U; ++j) acc[j] = finished(acc[j], old[j], p);
        if constexpr (VEC)
            store4(dst, acc);
        else
            store1(dst, acc[0]);
    }
}

// ---------------------------------------------------------------- few tokens
// At most this many tokens go without the sort.  Added to a 4000 x 2048 fp32 table, 23 tokens take 2.7 us
// and 512 5.7, where the sort's three launches take 17 for 513.  512 equal ids are the worst: one CTA
// a slab adds them all, 31 us against 19.
constexpr uint32_t kFewTokens = 512;
constexpr int kFewAhead = 16;  // rows loaded before they are added

struct FewParams {
    const void* ids;
    int32_t is64;
    uint32_t tokens;
    int64_t padding_id;
    uint32_t* status;
};

template <class DY, class DW, bool VEC>
__global__ void __launch_bounds__(kSumThreads) few_kernel(const FewParams f, const SumParams p, const DY* dy, DW* dw) {
    constexpr int U = VEC ? 8 : 1;
    constexpr int kWords = kFewTokens / 32;
    __shared__ uint32_t same[kWords];  // bit t: token t has this CTA's id
    __shared__ uint16_t list[kFewTokens];
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t mine = blockIdx.x;
    const int64_t id = load_id(f.ids, f.is64, mine);
    if (!takes_part(id, p.vocab, f.padding_id, f.status)) return;
#pragma unroll
    for (int w = warp; w < kWords; w += kSumThreads / 32) {
        const uint32_t t = w * 32 + lane;
        const uint32_t votes = __ballot_sync(0xffffffffu, t < f.tokens && load_id(f.ids, f.is64, t) == id);
        if (lane == 0) same[w] = votes;
    }
    __syncthreads();
    uint32_t n = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        if (w * 32 + 31 < mine ? same[w] != 0 : (w * 32 <= mine && (same[w] & ((1u << (mine & 31)) - 1)) != 0))
            return;  // an earlier token has the id: its CTA adds this row
        n += __popc(same[w]);
    }
    for (uint32_t t = threadIdx.x; t < f.tokens; t += kSumThreads) {
        if (!(same[t >> 5] >> (t & 31) & 1u)) continue;
        uint32_t at = __popc(same[t >> 5] & ((1u << (t & 31)) - 1));
        for (uint32_t w = 0; w < t >> 5; ++w) at += __popc(same[w]);
        list[at] = (uint16_t)t;
    }
    __syncthreads();
    const int64_t col = ((int64_t)blockIdx.y * kSumThreads + threadIdx.x) * U;
    if (col >= p.dim) return;
    DW* dst = dw + id * p.lddw + col;
    float acc[U] = {}, old[U] = {};
    if (p.accumulate) {
        if constexpr (VEC)
            unpack8(load8(dst), old);
        else
            old[0] = load1(dst);
    }
    for (uint32_t i0 = 0; i0 < n; i0 += kFewAhead) {
        Raw8<DY> raw[VEC ? kFewAhead : 1];
        float one[VEC ? 1 : kFewAhead];
#pragma unroll
        for (int a = 0; a < kFewAhead; ++a) {
            if (i0 + a >= n) break;
            const DY* src = dy + (int64_t)list[i0 + a] * p.lddy + col;
            if constexpr (VEC)
                raw[a] = load8(src);
            else
                one[a] = load1(src);
        }
#pragma unroll
        for (int a = 0; a < kFewAhead; ++a) {
            if (i0 + a >= n) break;
            if constexpr (VEC) {
                float v[8];
                unpack8(raw[a], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += v[j];
            } else {
                acc[0] += one[a];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) acc[j] = finished(acc[j], old[j], p);
    if constexpr (VEC)
        store8(dst, acc);
    else
        store1(dst, acc[0]);
}

// ---------------------------------------------------------------- launches
template <class DY, class DW, bool VEC>
cudaError_t launch_few(const FewParams& f, const SumParams& p, const void* dy, void* dw, cudaStream_t s) {
    constexpr int per = kSumThreads * (VEC ? 8 : 1);
    return launch_overlapped(few_kernel<DY, DW, VEC>, dim3(f.tokens, (unsigned)((p.dim + per - 1) / per)),
                             dim3(kSumThreads), 0, s, 1, true, f, p, static_cast<const DY*>(dy), static_cast<DW*>(dw));
}

template <class W, class Y, bool VEC>
cudaError_t launch_lookup(const void* ids, int is64, int64_t tokens, const void* w, int64_t vocab, int64_t dim,
                          int64_t ldw, float scale, void* y, int64_t ldy, cudaStream_t s) {
    const int64_t units = VEC ? dim / 8 : dim;
    const int64_t segs = (units + 32 * kLookupUnits - 1) / (32 * kLookupUnits);
    const int64_t blocks = (tokens * segs + kLookupThreads / 32 - 1) / (kLookupThreads / 32);
    if (blocks > INT32_MAX || segs > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_overlapped(lookup_kernel<W, Y, VEC>, dim3((unsigned)blocks), dim3(kLookupThreads), 0, s, 1, true, ids,
                             is64, tokens, static_cast<const W*>(w), vocab, dim, ldw, scale, static_cast<Y*>(y), ldy,
                             (uint32_t)segs, device_status_ptr());
}

cudaError_t sm_count(int* sms) {
    static DeviceSlots slots;
    return per_device_setting(slots, sms, [&](int dev, int* n) {
        return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
    });
}

template <class DY, class DW, bool VEC>
cudaError_t launch_sum(SumParams p, const void* dy, void* dw, int sms, cudaStream_t s) {
    constexpr int per = kSumThreads * (VEC ? 8 : 1);
    p.chunks = (p.tokens + kChunk - 1) / kChunk;
    const int64_t ctas = (int64_t)p.chunks * ((p.dim + per - 1) / per);
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto kern = p.accumulate ? sum_kernel<DY, DW, VEC, true> : sum_kernel<DY, DW, VEC, false>;
    cudaError_t e = launch_overlapped(kern, dim3((unsigned)ctas), dim3(kSumThreads), 0, s, 1, true, p,
                                      static_cast<const DY*>(dy), static_cast<DW*>(dw));
    if (e != cudaSuccess || p.chunks < 2) return e;
    constexpr int per_join = 32 * (VEC ? 4 : 1);
    const uint32_t slabs = (uint32_t)((p.dim + per_join - 1) / per_join);
    const int64_t most = (int64_t)(p.chunks - 1) * slabs;  // runs are at most one for each border
    return launch_overlapped(join_kernel<DW, VEC>, dim3((unsigned)std::min<int64_t>(most, 4 * sms)), dim3(kJoinThreads),
                             0, s, 1, true, p, static_cast<DW*>(dw), slabs);
}

template <int CTAS>
cudaError_t launch_sort_of(const SortParams& p, int sms, cudaStream_t s) {
    auto kern = sort_clear_kernel<CTAS>;
    static DeviceSlots slots;
    int set = 0;
    cudaError_t e = per_device_setting(slots, &set, [&](int, int* n) {
        *n = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
    });
    if (e != cudaSuccess) return e;
    const int64_t stretches = (p.rows * p.row_bytes + kClearBytes - 1) / kClearBytes;
    const int64_t clear_ctas = p.clear_flat ? stretches : std::min<int64_t>(stretches, 8 * sms);
    const int64_t clusters = 1 + ((p.clear ? clear_ctas : 0) + CTAS - 1) / CTAS;
    if (clusters * CTAS > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_overlapped(kern, dim3((unsigned)(clusters * CTAS)), dim3(kSortThreads), kSortSmem, s, CTAS, true, p);
}

cudaError_t launch_sort(const SortParams& p, int sms, cudaStream_t s) {
    if (p.tokens <= kSortTokens) return launch_sort_of<1>(p, sms, s);
    if (p.tokens <= 2 * kSortTokens) return launch_sort_of<2>(p, sms, s);
    if (p.tokens <= 4 * kSortTokens) return launch_sort_of<4>(p, sms, s);
    return launch_sort_of<kSortCtasMost>(p, sms, s);
}

bool valid_float(int t) { return t == MXFP4_OUT_F32 || t == MXFP4_OUT_BF16; }
int64_t esize(int t) { return t == MXFP4_OUT_BF16 ? 2 : 4; }
bool element_aligned(const void* p, int t) { return reinterpret_cast<uintptr_t>(p) % esize(t) == 0; }

constexpr int64_t kMaxDim = int64_t(1) << 20;  // the slabs of a few tokens fit in gridDim.y

int sort_passes(int64_t vocab) {
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;  // keys 0 .. vocab
    return (bits + kBits - 1) / kBits;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }
size_t sorted_bytes(int64_t tokens) { return up256((size_t)tokens * sizeof(uint2)); }
size_t chunks_of(int64_t tokens) { return (size_t)((tokens + kChunk - 1) / kChunk); }
// the number of runs (16 bytes) and the runs
size_t runs_bytes(int64_t tokens) { return up256(16 + chunks_of(tokens) * sizeof(Run)); }

// Whether the grids of a call's launches hold: tokens x slabs of the narrowest kind (single elements).
bool grids_fit(int64_t tokens, int64_t dim) {
    return tokens * ((dim + kSumThreads - 1) / kSumThreads) / 8 < INT32_MAX / 4;
}

mxfp4_status check_table(const char* what, int ids_dtype, int64_t tokens, int64_t vocab, int64_t dim) {
    if (ids_dtype != MXFP4_IDS_I32 && ids_dtype != MXFP4_IDS_I64)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad ids_dtype %d", what, ids_dtype);
    if (tokens < 0 || vocab < 0 || dim < 0) return record_error(MXFP4_ERR_INVALID_ARG, "%s: negative size", what);
    if (tokens > INT32_MAX || vocab >= INT32_MAX || dim > kMaxDim)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: tokens and vocab must be below 2^31, dim at most %lld",
                            what, (long long)kMaxDim);
    if (!grids_fit(tokens, dim))
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: %lld tokens of %lld columns are too many", what,
                            (long long)tokens, (long long)dim);
    return MXFP4_OK;
}

// A typed pointer with a leading dimension: non-NULL, aligned to its element, ld >= dim.
mxfp4_status check_matrix(const char* what, const char* name, const void* p, int dtype, int64_t dim, int64_t ld) {
    if (!valid_float(dtype)) return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad dtype %d of %s", what, dtype, name);
    if (!p) return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s is NULL", what, name);
    if (!element_aligned(p, dtype))
        return record_error(MXFP4_ERR_MISALIGNED, "%s: %s not aligned to its element type", what, name);
    if (ld < dim) return record_error(MXFP4_ERR_INVALID_ARG, "%s: leading dimension of %s below dim", what, name);
    return MXFP4_OK;
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" mxfp4_status mxfp4_embedding(const void* ids, int ids_dtype, int64_t tokens, const void* w, int w_dtype,
                                        int64_t vocab, int64_t dim, int64_t ldw, float scale, void* y, int y_dtype,
                                        int64_t ldy, mxfp4_stream_t stream) {
    const char* what = "embedding";
    mxfp4_status st = check_table(what, ids_dtype, tokens, vocab, dim);
    if (st) return st;
    if (!valid_float(w_dtype) || !valid_float(y_dtype))
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad dtype (%d, %d)", what, w_dtype, y_dtype);
    if (tokens == 0 || dim == 0) return record_error(MXFP4_OK, "%s", "");
    if (vocab == 0) return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: an empty table", what);
    if (!ids) return record_error(MXFP4_ERR_INVALID_ARG, "%s: ids is NULL", what);
    if (reinterpret_cast<uintptr_t>(ids) % (ids_dtype == MXFP4_IDS_I64 ? 8 : 4))
        return record_error(MXFP4_ERR_MISALIGNED, "%s: ids not aligned to their type", what);
    if ((st = check_matrix(what, "w", w, w_dtype, dim, ldw))) return st;
    if ((st = check_matrix(what, "y", y, y_dtype, dim, ldy))) return st;
    if ((st = ensure_device())) return st;
    const bool vec = vector_rows(w, ldw, dim, esize(w_dtype)) && vector_rows(y, ldy, dim, esize(y_dtype));
    const int is64 = ids_dtype == MXFP4_IDS_I64;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto wt, auto yt) {
        using W = decltype(wt);
        using Y = decltype(yt);
        return vec ? launch_lookup<W, Y, true>(ids, is64, tokens, w, vocab, dim, ldw, scale, y, ldy, s)
                   : launch_lookup<W, Y, false>(ids, is64, tokens, w, vocab, dim, ldw, scale, y, ldy, s);
    };
    const bool wb = w_dtype == MXFP4_OUT_BF16, yb = y_dtype == MXFP4_OUT_BF16;
    const cudaError_t e = wb ? (yb ? go(bf16{}, bf16{}) : go(bf16{}, float{})) : (yb ? go(float{}, bf16{}) : go(float{}, float{}));
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}

extern "C" size_t mxfp4_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
    if (tokens <= 0 || vocab <= 0 || dim <= 0 || tokens > INT32_MAX || vocab >= INT32_MAX || dim > kMaxDim) return 0;
    return 2 * sorted_bytes(tokens) + runs_bytes(tokens) + up256(chunks_of(tokens) * 2 * (size_t)dim * sizeof(float));
}

extern "C" mxfp4_status mxfp4_embedding_grad(const void* ids, int ids_dtype, int64_t tokens, const void* dy,
                                             int dy_dtype, int64_t lddy, int64_t vocab, int64_t dim, float scale,
                                             int64_t padding_id, void* dw, int dw_dtype, int64_t lddw, int accumulate,
                                             void* ws, size_t ws_bytes, mxfp4_stream_t stream) {
    const char* what = "embedding_grad";
    mxfp4_status st = check_table(what, ids_dtype, tokens, vocab, dim);
    if (st) return st;
    if (!valid_float(dy_dtype) || !valid_float(dw_dtype))
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad dtype (%d, %d)", what, dy_dtype, dw_dtype);
    if (accumulate != 0 && accumulate != 1)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: accumulate must be 0 or 1", what);
    if (vocab == 0 || dim == 0) return record_error(MXFP4_OK, "%s", "");
    if ((st = check_matrix(what, "dw", dw, dw_dtype, dim, lddw))) return st;
    if (tokens > 0) {
        if (!ids) return record_error(MXFP4_ERR_INVALID_ARG, "%s: ids is NULL", what);
        if (reinterpret_cast<uintptr_t>(ids) % (ids_dtype == MXFP4_IDS_I64 ? 8 : 4))
            return record_error(MXFP4_ERR_MISALIGNED, "%s: ids not aligned to their type", what);
        if ((st = check_matrix(what, "dy", dy, dy_dtype, dim, lddy))) return st;
        const size_t need = mxfp4_embedding_grad_workspace_bytes(tokens, vocab, dim);
        if (!ws || ws_bytes < need)
            return record_error(MXFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", what, need);
        if (reinterpret_cast<uintptr_t>(ws) % 256)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: workspace not 256-byte aligned", what);
    } else if (accumulate) {
        return record_error(MXFP4_OK, "%s", "");
    }
    if ((st = ensure_device())) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t wsz = esize(dw_dtype);

    SortParams sp{};
    sp.ids = ids;
    sp.is64 = ids_dtype == MXFP4_IDS_I64;
    const bool few = tokens <= kFewTokens;
    sp.passes = few ? 0 : sort_passes(vocab);
    sp.tokens = few ? 0 : (uint32_t)tokens;
    sp.vocab = vocab;
    sp.padding_id = padding_id;
    uint8_t* at = static_cast<uint8_t*>(ws);
    sp.buf[0] = reinterpret_cast<uint2*>(at);
    sp.buf[1] = tokens > 0 ? reinterpret_cast<uint2*>(at + sorted_bytes(tokens)) : nullptr;
    if (tokens > 0) {
        sp.num_runs = reinterpret_cast<uint32_t*>(at + 2 * sorted_bytes(tokens));
    }
    sp.status = device_status_ptr();
    sp.dw = static_cast<uint8_t*>(dw);
    sp.rows = vocab;
    sp.row_bytes = dim * wsz;
    sp.pitch_bytes = lddw * wsz;
    const bool base16 = reinterpret_cast<uintptr_t>(dw) % 16 == 0;
    sp.clear_flat = base16 && sp.pitch_bytes == sp.row_bytes;
    sp.clear_vec = base16 && sp.row_bytes % 16 == 0 && sp.pitch_bytes % 16 == 0;
    sp.clear = !accumulate;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess && !(few && accumulate)) e = launch_sort(sp, sms, s);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s sort launch: %s", what, cudaGetErrorString(e));
    if (tokens == 0) return record_error(MXFP4_OK, "%s", "");

    SumParams p{};
    p.sorted = sp.buf[0];
    p.tokens = (uint32_t)tokens;
    p.vocab = vocab;
    p.dim = dim;
    p.lddy = lddy;
    p.lddw = lddw;
    p.scale = scale;
    p.accumulate = accumulate;
    p.runs = reinterpret_cast<Run*>(at + 2 * sorted_bytes(tokens) + 16);
    p.num_runs = sp.num_runs;
    p.part = reinterpret_cast<float*>(at + 2 * sorted_bytes(tokens) + runs_bytes(tokens));
    const bool vec = vector_rows(dy, lddy, dim, esize(dy_dtype)) && vector_rows(dw, lddw, dim, wsz);
    const FewParams fp{ids, sp.is64, (uint32_t)tokens, padding_id, sp.status};
    auto go = [&](auto yt, auto wt) {
        using DY = decltype(yt);
        using DW = decltype(wt);
        if (few) return vec ? launch_few<DY, DW, true>(fp, p, dy, dw, s) : launch_few<DY, DW, false>(fp, p, dy, dw, s);
        return vec ? launch_sum<DY, DW, true>(p, dy, dw, sms, s) : launch_sum<DY, DW, false>(p, dy, dw, sms, s);
    };
    const bool yb = dy_dtype == MXFP4_OUT_BF16, wb = dw_dtype == MXFP4_OUT_BF16;
    e = yb ? (wb ? go(bf16{}, bf16{}) : go(bf16{}, float{})) : (wb ? go(float{}, bf16{}) : go(float{}, float{}));
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}
