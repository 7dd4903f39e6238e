// rope.cu -- norm of each head of queries and keys with the rotation by position in the same pass, and its gradient.
//
//   r = 1 / sqrt(mean x^2 + eps),  n = x r gain          (no gain: n = x)
//   (a, b) -> (a cos - b sin, b cos + a sin),  angle = positions[axis of the pair][token] * freq[pair]
// Backwards, with dz the gradient turned back by the same angles and u = x r:
//   dx = r (dz gain - u mean(dz gain u)),   dgain = sum over tokens and heads of dz u
//
// HBM bandwidth bounds long calls, latency short ones.  A warp takes a token, or a share of its heads where there are few
// tokens: it makes the cosines and sines of the token's pairs once for all heads (shared memory of its own, no barrier of
// the block), then goes through the heads of queries and of keys.  Groups of lanes hold a row (a token's head) each, a lane
// VEC pairs of it, as two runs of VEC elements (or one of 2 VEC, where a pair's elements are neighbours), with turn and gain
// in registers; the loads of ROWS rows are under way together, and in long calls (STAGED) the next ROWS are on their way
// to shared memory while these are worked on.  Every row is read once and written once.  The elements behind the rotated ones
// are pairs that do not turn.  8192 tokens of 32 and 8 heads of 128: 33.7 us for 168 MB, backwards 56.9 us for 252 MB; a
// plain copy of as much takes 28.8 us, and a sum of two tensors into a third 39.1.  Backwards neither the issue slots (58%) nor
// HBM (65%) are what bounds it but the warps' own chains, 16 of them an SM: of 6.5 cycles for an instruction 1.7 are fixed
// latencies, 1.1 lanes' exchange and shared memory, 0.5 loads.
//
// Angles.  A position times a frequency in fp32 is off by 2^-24 of itself, which is 0.03 radians at position 500000.  Here a
// frequency is held as turns per position in 64-bit fixed point, and a product with an integer modulo 2^64 is the exact
// fraction of a turn: what is left is the frequency's own rounding (2^-65 turns a position), whatever the position.
#include <algorithm>
#include <cmath>

#include "element.cuh"
#include "heads.cuh"
#include "quant_math.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kRopeThreads = 256;
constexpr int kWarps = kRopeThreads / 32;
constexpr int kMaxHeadDim = 256;
constexpr int kMaxPairs = kMaxHeadDim / 2;

struct RopeSide {  // queries or keys
    const void* x;
    const void* dy;  // gradient only
    void* y;         // the result: y, or dx
    int64_t x_token, x_head, dy_token, dy_head, y_token, y_head;  // bytes
    int32_t heads;
    const float* gain;
};

struct RopeParams {
    RopeSide side[2];
    int32_t tokens, dim, pairs, is64;
    int32_t interleaved;
    int32_t span;    // slices of heads that a warp takes of a token
    int64_t items;   // tokens times shares of their slices
    float eps;
    const void* positions;  // [axes][tokens]
    float* partial;         // gradient only: [CTA][2][dim]
    uint64_t freq[kMaxPairs];
    uint8_t axis[kMaxPairs];
};

// VEC neighbouring elements as they lie in memory, aligned to their size in bytes (at most 32).
template <class T, int VEC>
struct Run {
    T v[VEC];
};
template <>
struct __align__(16) Run<float, 4> {
    float v[4];
};
template <>
struct Run<bf16, 8> {
    uint4 w;
};
template <>
struct Run<bf16, 4> {
    uint2 w;
};
template <class T, int VEC>
__device__ __forceinline__ void load_run(const T* p, Run<T, VEC>& r) {
    if constexpr (sizeof(T) == 2 && VEC >= 4) {
        r.w = *reinterpret_cast<const decltype(r.w)*>(p);
    } else if constexpr (VEC == 4) {
        load4(p, r.v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = p[i];
    }
}
template <int VEC>
__device__ __forceinline__ void unpack_run(const Run<float, VEC>& r, float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r.v[i];
}
template <int VEC>
__device__ __forceinline__ void unpack_run(const Run<bf16, VEC>& r, float (&v)[VEC]) {
    if constexpr (VEC >= 4) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r.w);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __bfloat162float(r.v[i]);
    }
}
template <int VEC, class T>
__device__ __forceinline__ void store_run(T* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8)
        store8(p, v);
    else if constexpr (VEC == 4)
        store4(p, v);
    else
#pragma unroll
        for (int i = 0; i < VEC; ++i) store1(p + i, v[i]);
}

// VEC pairs from a row's two runs: a[i], b[i].
template <bool NEIGHBOURS, class T, int VEC>
__device__ __forceinline__ void pairs_of(const Run<T, VEC>& ru, const Run<T, VEC>& rv, float (&a)[VEC], float (&b)[VEC]) {
    float u[2 * VEC];
    unpack_run<VEC>(ru, *reinterpret_cast<float(*)[VEC]>(u));
    unpack_run<VEC>(rv, *reinterpret_cast<float(*)[VEC]>(u + VEC));
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = u[NEIGHBOURS ? 2 * i : i], b[i] = u[NEIGHBOURS ? 2 * i + 1 : VEC + i];
}
template <bool NEIGHBOURS, int VEC, class T>
__device__ __forceinline__ void store_pairs(T* row, int at_a, int at_b, const float (&a)[VEC], const float (&b)[VEC]) {
    float u[2 * VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) u[NEIGHBOURS ? 2 * i : i] = a[i], u[NEIGHBOURS ? 2 * i + 1 : VEC + i] = b[i];
    store_run<VEC>(row + at_a, *reinterpret_cast<float(*)[VEC]>(u));
    store_run<VEC>(row + at_b, *reinterpret_cast<float(*)[VEC]>(u + VEC));
}

// N neighbouring floats of shared memory, aligned to their size (16 bytes at most).
template <int N>
__device__ __forceinline__ void load_shared(const float* p, float (&v)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 w = *reinterpret_cast<const float4*>(p + i);
            v[i] = w.x, v[i + 1] = w.y, v[i + 2] = w.z, v[i + 3] = w.w;
        }
    } else if constexpr (N == 2) {
        const float2 w = *reinterpret_cast<const float2*>(p);
        v[0] = w.x, v[1] = w.y;
    } else {
        v[0] = p[0];
    }
}

// d = a b + c and the like on N numbers, two in an instruction.
template <int N>
__device__ __forceinline__ void mul_n(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
    if constexpr (N == 1) d[0] = a[0] * b[0];
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 r = f2_mul(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
        d[i] = r.x, d[i + 1] = r.y;
    }
}
template <int N>
__device__ __forceinline__ void fma_n(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
    if constexpr (N == 1) d[0] = fmaf(a[0], b[0], c[0]);
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 r = f2_fma(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
        d[i] = r.x, d[i + 1] = r.y;
    }
}
template <int N>
__device__ __forceinline__ void scale_n(float (&d)[N], const float (&a)[N], float by) {
    float b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = by;
    mul_n(d, a, b);
}
template <int N>
__device__ __forceinline__ float sum_n(const float (&a)[N]) {
    float v = a[0];
#pragma unroll
    for (int i = 1; i < N; ++i) v += a[i];
    return v;
}

// Sums of N numbers over the `n` lanes of a row's group, in every one of them (li: this lane's place in it).
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int li, int n) {
    if ((n & (n - 1)) == 0) {  // groups start on their own size
        for (int o = n >> 1; o > 0; o >>= 1) {
            float w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += w[i];
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    for (int o = 1 << (31 - __clz(n - 1)); o > 0; o >>= 1) {
        float w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __shfl_down_sync(0xffffffffu, v[i], o);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (li < o && li + o < n) v[i] += w[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], lane - li);
}

// A run's way from global to shared memory without registers, and the wait for all but the last `N` groups of them.
template <class R>
__device__ __forceinline__ void copy_run(R* to, const void* from) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (sizeof(R) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(sizeof(R)) : "memory");
}
__device__ __forceinline__ void end_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Lanes of a row, and rows that a warp takes at once.
__host__ __device__ inline int row_lanes(int half, int vec) { return half / vec < 32 ? half / vec : 32; }

// Runs that a thread holds in shared memory for a slice of heads, of x, and of dy in the gradient.
__host__ __device__ constexpr int staged_runs(bool staged, int rows, bool grad) { return staged ? rows * (grad ? 2 : 1) * 2 : 0; }
constexpr int kStages = 2;
// Slices that a warp must have to go through for the next one's copies to be worth their instructions.  32 and 8 heads of
// 128, with them and without: 16384 tokens 57.5 and 61.9 us, gradient 109 and 113; 8192 tokens 34.3 and 37.1, 59.6 and 64.5;
// 4096 tokens (5 and 8 slices) 20.3 and 18.7, 39.1 and 39.2; 512 tokens 10.4 and 8.4, 16.5 and 14.6.  Calls in fp32 lose
// at 5003 tokens of 14 and 2 heads of 72 (20.7 and 18.6, 33.0 and 28.8) and are left without.
constexpr int kStagedSlices = 10;

// SLOTS: runs of pairs of a lane, 32 lanes apart (rows of more than 32 VEC pairs).  ROWS: that a lane has under way.
template <class T, int VEC, int SLOTS, int ROWS, bool NEIGHBOURS, bool GRAD, bool STAGED>
__global__ void __launch_bounds__(kRopeThreads, GRAD ? 2 : VEC * SLOTS >= 8 ? 2 : 3)
    rope_kernel(const __grid_constant__ RopeParams p) {
    static_assert(!STAGED || SLOTS == 1);
    constexpr int kRuns = staged_runs(STAGED, ROWS, GRAD);
    extern __shared__ __align__(16) uint8_t staged[];
    constexpr int kSums = GRAD ? kRopeThreads * 2 * VEC * SLOTS : 0;  // floats of the groups' sums of gains
    constexpr int kTurn = kWarps * kMaxPairs * 2;
    __shared__ __align__(16) float shared[kTurn + 2 * kMaxHeadDim > kSums ? kTurn + 2 * kMaxHeadDim : kSums];
    const int half = p.dim / 2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2* turn = reinterpret_cast<float2*>(shared) + warp * kMaxPairs;
    float* gains = shared + kTurn;
    const int lanes = row_lanes(half, VEC), per_warp = 32 / lanes;
    const bool idle = lane >= lanes * per_warp;
    const int li = lane % lanes, sub = lane / lanes;
    // where this lane's elements are; a run that is past the row is the first one's again, not counted and not written
    int at_a[SLOTS], at_b[SLOTS], pair[SLOTS];
    bool there[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        there[s] = (li + s * lanes) * VEC < half;
        const int c = there[s] ? (li + s * lanes) * VEC : 0;  // first pair
        pair[s] = c;
        if (NEIGHBOURS) {
            at_a[s] = 2 * c, at_b[s] = 2 * c + VEC;
        } else if (c < p.pairs) {
            at_a[s] = c, at_b[s] = c + p.pairs;
        } else {
            at_a[s] = p.pairs + c, at_b[s] = half + c;
        }
    }
    auto element = [&](int s, int which, int i) {  // of pair i of slot s in its row
        return NEIGHBOURS ? at_a[s] + 2 * i + which : (which ? at_b[s] : at_a[s]) + i;
    };
    const int slice = per_warp * ROWS;  // heads
    const int slices0 = (p.side[0].heads + slice - 1) / slice;
    const int all = slices0 + (p.side[1].heads + slice - 1) / slice, shares = (all + p.span - 1) / p.span;
    const int64_t first_item = (int64_t)blockIdx.x * kWarps + warp, step = (int64_t)gridDim.x * kWarps;
    // The slice that is copied next, and the stage that it goes to.
    int64_t next_item = first_item, next_token;
    int next, next_end, next_stage = 0;
    auto share_of = [&](int64_t item, int64_t& token, int& from, int& to) {
        token = shares == 1 ? item : item / shares;
        from = (int)(item - token * shares) * p.span, to = min(from + p.span, all);
    };
    share_of(next_item, next_token, next, next_end);
    auto run_at = [&](int stage, int i) {
        return reinterpret_cast<Run<T, VEC>*>(staged) + (stage * kRuns + i) * kRopeThreads + threadIdx.x;
    };
    auto copy_next = [&] {
        if (next_item < p.items) {
            const int which = next >= slices0;
            const RopeSide& side = p.side[which];
            const char* rows_x = static_cast<const char*>(side.x) + next_token * side.x_token;
            const char* rows_dy = static_cast<const char*>(side.dy) + next_token * side.dy_token;
            const int h0 = (which ? next - slices0 : next) * slice + sub;
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const uint32_t h = h0 + k * per_warp;
                if (h >= (uint32_t)side.heads || idle) continue;
                if (!GRAD || side.gain) {
                    const T* row = reinterpret_cast<const T*>(rows_x + h * side.x_head);
                    copy_run(run_at(next_stage, 2 * k), row + at_a[0]);
                    copy_run(run_at(next_stage, 2 * k + 1), row + at_b[0]);
                }
                if constexpr (GRAD) {
                    const T* row = reinterpret_cast<const T*>(rows_dy + h * side.dy_head);
                    copy_run(run_at(next_stage, 2 * (ROWS + k)), row + at_a[0]);
                    copy_run(run_at(next_stage, 2 * (ROWS + k) + 1), row + at_b[0]);
                }
            }
            if (++next == next_end) {
                next_item += step;
                share_of(next_item, next_token, next, next_end);
            }
            next_stage ^= 1;
        }
        end_copies();
    };
    int stage = 0;
    grid_dependency_wait();
    allow_dependent_launch();
    if constexpr (STAGED) copy_next();
    for (int i = threadIdx.x; i < 2 * p.dim; i += kRopeThreads) {
        const float* gain = p.side[i >= p.dim].gain;
        gains[i] = gain ? gain[i >= p.dim ? i - p.dim : i] : 1.f;
    }
    __syncthreads();
    float dgain[2][SLOTS][2][VEC] = {};
    const float mean = 1.f / (float)p.dim;
    for (int64_t item = first_item; item < p.items; item += step) {
        int64_t token;
        int first, end;
        share_of(item, token, first, end);
        __syncwarp();  // the cosines of the token before have been read
        for (int i = lane; i < half; i += 32) {
            float2 cs = make_float2(1.f, 0.f);
            if (i < p.pairs) {
                const int64_t pos = load_id(p.positions, p.is64, (int64_t)p.axis[i] * p.tokens + token);
                const int64_t frac = (int64_t)((uint64_t)pos * p.freq[i]);  // of a turn, times 2^64
                sincospif((float)(int32_t)(frac >> 32) * 0x1p-31f, &cs.y, &cs.x);
            }
            turn[i] = cs;
        }
        __syncwarp();
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const RopeSide& side = p.side[which];
            const bool norm = side.gain != nullptr;
            const int from = which ? max(first - slices0, 0) : first, to = which ? end - slices0 : min(end, slices0);
            if (from >= to) continue;
            // forward: (a, b) -> (a ca - b sb, b cb + a sa), the gains in the factors; backward: the turn alone
            float ca[SLOTS][VEC], sa[SLOTS][VEC], cb[GRAD ? 1 : SLOTS][VEC], sb[SLOTS][VEC], gain[GRAD ? SLOTS : 1][2][VEC];
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                float cs[2 * VEC], ga[VEC], gb[VEC], g[2 * VEC];
                load_shared(reinterpret_cast<const float*>(turn + pair[s]), cs);
                if (NEIGHBOURS) {
                    load_shared(gains + which * p.dim + at_a[s], g);
                } else {
                    load_shared(gains + which * p.dim + at_a[s], *reinterpret_cast<float(*)[VEC]>(g));
                    load_shared(gains + which * p.dim + at_b[s], *reinterpret_cast<float(*)[VEC]>(g + VEC));
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    ga[i] = g[NEIGHBOURS ? 2 * i : i], gb[i] = g[NEIGHBOURS ? 2 * i + 1 : VEC + i];
                    if constexpr (GRAD) {
                        ca[s][i] = cs[2 * i], sa[s][i] = cs[2 * i + 1], sb[s][i] = -cs[2 * i + 1];
                        gain[s][0][i] = ga[i], gain[s][1][i] = gb[i];
                    } else {
                        ca[s][i] = cs[2 * i] * ga[i], sa[s][i] = cs[2 * i + 1] * ga[i];
                        cb[s][i] = cs[2 * i] * gb[i], sb[s][i] = -cs[2 * i + 1] * gb[i];
                    }
                }
            }
            const char* rows_x = static_cast<const char*>(side.x) + token * side.x_token;
            const char* rows_dy = static_cast<const char*>(side.dy) + token * side.dy_token;
            char* rows_y = static_cast<char*>(side.y) + token * side.y_token;
            for (int h0 = from * slice; h0 < min(to * slice, side.heads); h0 += slice) {
                Run<T, VEC> x[ROWS][SLOTS][2], dy[GRAD ? ROWS : 1][SLOTS][2];
                int h[ROWS];
                if constexpr (STAGED) {
                    copy_next();
                    wait_copies<kStages - 1>();  // a lane reads what it copied itself
#pragma unroll
                    for (int k = 0; k < ROWS; ++k) {
                        h[k] = idle ? side.heads : h0 + k * per_warp + sub;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            x[k][0][i] = *run_at(stage, 2 * k + i);
                            if constexpr (GRAD) dy[k][0][i] = *run_at(stage, 2 * (ROWS + k) + i);
                        }
                    }
                    stage ^= 1;
                } else {
                    // Lanes without a row of their own read the last head's, and write nothing.
#pragma unroll
                    for (int k = 0; k < ROWS; ++k) {
                        if (k > 0 && k % 2 == 0 && h0 + k * per_warp >= side.heads) break;
                        h[k] = h0 + k * per_warp + sub;
                        const uint32_t at = min(h[k], side.heads - 1);
                        const T* px = reinterpret_cast<const T*>(rows_x + at * side.x_head);
                        const T* pd = reinterpret_cast<const T*>(rows_dy + at * side.dy_head);
#pragma unroll
                        for (int s = 0; s < SLOTS; ++s) {
                            if (!GRAD || norm) {
                                load_run<T, VEC>(px + at_a[s], x[k][s][0]);
                                load_run<T, VEC>(px + at_b[s], x[k][s][1]);
                            }
                            if constexpr (GRAD) {
                                load_run<T, VEC>(pd + at_a[s], dy[k][s][0]);
                                load_run<T, VEC>(pd + at_b[s], dy[k][s][1]);
                            }
                        }
                        if (idle) h[k] = side.heads;
                    }
                }
                // two rows together, so that one's sum over lanes is under way while the other's is
#pragma unroll
                for (int k0 = 0; k0 < ROWS; k0 += 2) {
                    if (k0 > 0 && h0 + k0 * per_warp >= side.heads) break;
                    float a[2][SLOTS][VEC], b[2][SLOTS][VEC], u[2][SLOTS][VEC], v[2][SLOTS][VEC];
                    float sums[GRAD ? 4 : 2];  // of x x; and of dz gain x, which needs no norm yet: one trip over the lanes
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float ss[VEC] = {}, dot[VEC] = {};
#pragma unroll
                        for (int s = 0; s < SLOTS; ++s) {
                            if (!GRAD || norm) {
                                pairs_of<NEIGHBOURS, T, VEC>(x[k0 + r][s][0], x[k0 + r][s][1], a[r][s], b[r][s]);
                                if (SLOTS == 1 || there[s]) {
                                    fma_n(ss, a[r][s], a[r][s], ss);
                                    fma_n(ss, b[r][s], b[r][s], ss);
                                }
                            }
                            if constexpr (GRAD) {  // dz
                                float da[VEC], db[VEC];
                                pairs_of<NEIGHBOURS, T, VEC>(dy[k0 + r][s][0], dy[k0 + r][s][1], da, db);
                                mul_n(u[r][s], da, ca[s]);
                                mul_n(v[r][s], db, ca[s]);
                                fma_n(u[r][s], db, sa[s], u[r][s]);
                                fma_n(v[r][s], da, sb[s], v[r][s]);
                                if (norm && (SLOTS == 1 || there[s])) {
                                    float zx[VEC];
                                    mul_n(zx, u[r][s], a[r][s]);
                                    fma_n(dot, zx, gain[s][0], dot);
                                    mul_n(zx, v[r][s], b[r][s]);
                                    fma_n(dot, zx, gain[s][1], dot);
                                }
                            }
                        }
                        sums[r] = sum_n(ss);
                        if constexpr (GRAD) sums[2 + r] = sum_n(dot);
                    }
                    if (norm) group_sums(sums, li, lanes);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float rstd = norm ? rsqrtf(fmaf(sums[r], mean, p.eps)) : 1.f;
                        if constexpr (!GRAD) {
#pragma unroll
                            for (int s = 0; s < SLOTS; ++s) {
                                mul_n(u[r][s], a[r][s], ca[s]);
                                mul_n(v[r][s], b[r][s], cb[s]);
                                fma_n(u[r][s], b[r][s], sb[s], u[r][s]);
                                fma_n(v[r][s], a[r][s], sa[s], v[r][s]);
                                if (norm) {
                                    scale_n(u[r][s], u[r][s], rstd);
                                    scale_n(v[r][s], v[r][s], rstd);
                                }
                            }
                        } else if (norm) {
                            // rows that are another lane's, and runs that are no lane's, add nothing to the gains' sums
                            const bool mine = h[k0 + r] < side.heads;
                            // (dz gain - u mean(dz gain u)) r with u = x r
                            const float along = -sums[2 + r] * mean * rstd * rstd;
                            float by[VEC];
#pragma unroll
                            for (int i = 0; i < VEC; ++i) by[i] = along;
#pragma unroll
                            for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                                for (int w = 0; w < 2; ++w) {
                                    float(&x1)[VEC] = w ? b[r][s] : a[r][s];
                                    float(&dz)[VEC] = w ? v[r][s] : u[r][s];
                                    float ux[VEC];
                                    if (mine && (SLOTS == 1 || there[s])) {
                                        scale_n(ux, x1, rstd);
                                        fma_n(dgain[which][s][w], dz, ux, dgain[which][s][w]);
                                    }
                                    mul_n(dz, dz, gain[s][w]);
                                    fma_n(dz, x1, by, dz);
                                    scale_n(dz, dz, rstd);
                                }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (h[k0 + r] < side.heads) {
                            T* py = reinterpret_cast<T*>(rows_y + (uint32_t)h[k0 + r] * side.y_head);
#pragma unroll
                            for (int s = 0; s < SLOTS; ++s)
                                if (SLOTS == 1 || there[s])
                                    store_pairs<NEIGHBOURS, VEC>(py, at_a[s], at_b[s], u[r][s], v[r][s]);
                        }
                }
            }
        }
    }
    if constexpr (GRAD) {
        if (!p.partial) return;
        // the groups' sums, added up in their order
        const int groups = kWarps * per_warp;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            if (!idle) {
                float* at = shared + (warp * per_warp + sub) * p.dim;
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (there[s]) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
#pragma unroll
                            for (int w = 0; w < 2; ++w) at[element(s, w, i)] = dgain[which][s][w][i];
                    }
            }
            __syncthreads();
            for (int d = threadIdx.x; d < p.dim; d += kRopeThreads) {
                float v = 0.f;
                for (int g = 0; g < groups; ++g) v += shared[g * p.dim + d];
                p.partial[((int64_t)blockIdx.x * 2 + which) * p.dim + d] = v;
            }
        }
    }
}

// dgain[d] of one side: the CTAs' sums, 32 threads of a column each adding up every 32nd, then those in their order.
__global__ void __launch_bounds__(1024) rope_gain_kernel(const float* partial, int ctas, int dim, float* q_dgain,
                                                         float* k_dgain) {
    __shared__ float sums[32][33];
    grid_dependency_wait();
    allow_dependent_launch();
    const int column = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + column, which = blockIdx.y;
    float v = 0.f;
    if (d < dim)
        for (int c = part; c < ctas; c += 32) v += partial[((int64_t)c * 2 + which) * dim + d];
    sums[part][column] = v;
    __syncthreads();
    if (part == 0 && d < dim) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += sums[i][column];
        float* out = which ? k_dgain : q_dgain;
        if (out) out[d] = v;
    }
}

cudaError_t sm_count(int* sms) {
    static DeviceSlots slots;
    return per_device_setting(slots, sms, [](int dev, int* v) {
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
    });
}

constexpr int kMaxCtas = 1024;  // bounds the gradient's workspace

// Launches the kernel over `ctas` CTAs at most: a warp for each token, or for each share of a token's heads where there are
// fewer tokens than warps.
template <class T, int VEC, int SLOTS, int ROWS, bool NEIGHBOURS, bool GRAD, bool STAGED = false>
cudaError_t launch_shares(RopeParams p, int sms, int* ctas, cudaStream_t s) {
    const int slice = 32 / row_lanes(p.dim / 2, VEC) * ROWS;
    int all = 0;
    for (const RopeSide& side : p.side) all += (side.heads + slice - 1) / slice;
    const int most = std::min(kMaxCtas, sms * (GRAD ? 2 : VEC * SLOTS >= 8 ? 2 : 3));  // that fit the device at once
    const int64_t warps = (int64_t)most * kWarps;
    if constexpr (sizeof(T) == 2 && VEC == (GRAD ? 4 : 8) && !STAGED)
        if ((int64_t)p.tokens * all >= kStagedSlices * warps)
            return launch_shares<T, VEC, SLOTS, ROWS, NEIGHBOURS, GRAD, true>(p, sms, ctas, s);
    p.span = (int32_t)std::min<int64_t>(all, std::max<int64_t>(1, (int64_t)p.tokens * all / warps));
    p.items = (int64_t)p.tokens * ((all + p.span - 1) / p.span);
    *ctas = (int)std::min<int64_t>(most, (p.items + kWarps - 1) / kWarps);
    const auto kernel = rope_kernel<T, VEC, SLOTS, ROWS, NEIGHBOURS, GRAD, STAGED>;
    const int smem = kStages * staged_runs(STAGED, ROWS, GRAD) * kRopeThreads * (int)sizeof(Run<T, VEC>);
    static DeviceSlots ready;
    int unused = 0;
    const cudaError_t e = per_device_setting(ready, &unused, [&](int, int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, dim3((unsigned)*ctas), dim3(kRopeThreads), (size_t)smem, s, 1, true, p);
}
template <class T, bool NEIGHBOURS, bool GRAD>
cudaError_t launch_rope(const RopeParams& p, int vec, int sms, int* ctas, cudaStream_t s) {
    if constexpr (!GRAD && sizeof(T) == 2)
        if (vec == 8) return launch_shares<T, 8, 1, 4, NEIGHBOURS, false>(p, sms, ctas, s);
    if (vec >= 4) return launch_shares<T, 4, 1, GRAD && sizeof(T) == 4 ? 2 : 4, NEIGHBOURS, GRAD>(p, sms, ctas, s);
    if (vec == 2) return launch_shares<T, 2, 2, 2, NEIGHBOURS, GRAD>(p, sms, ctas, s);
    return launch_shares<T, 1, 4, 2, NEIGHBOURS, GRAD>(p, sms, ctas, s);
}
template <bool GRAD>
cudaError_t launch_rope(const RopeParams& p, int dtype, int vec, int sms, int* ctas, cudaStream_t s) {
    if (dtype == MXFP4_OUT_BF16)
        return p.interleaved ? launch_rope<bf16, true, GRAD>(p, vec, sms, ctas, s)
                             : launch_rope<bf16, false, GRAD>(p, vec, sms, ctas, s);
    return p.interleaved ? launch_rope<float, true, GRAD>(p, vec, sms, ctas, s)
                         : launch_rope<float, false, GRAD>(p, vec, sms, ctas, s);
}

// Radians per position as the fraction of a turn in 64-bit fixed point, with 1 / (2 pi) as the sum of two doubles.
uint64_t fixed_turns(double x) {
    const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    const double a = std::fabs(x), t = a * hi, rest = std::fma(a, hi, -t) + a * lo;
    uint64_t v = (uint64_t)std::ldexp(t - std::floor(t), 64);   // exact: below 2^64, a double's 53 bits
    v += (uint64_t)(int64_t)std::llrint(std::ldexp(rest, 64));  // below 2^30 for |x| up to 1e6
    return x < 0 ? 0 - v : v;
}

// What both directions share: checks, and the parameters that do not depend on the direction.
mxfp4_status rope_common(const char* what, int64_t tokens, int64_t dim, float eps, const mxfp4_rope* rope,
                         const void* positions, int ids_dtype, int64_t axes, RopeParams* p) {
    if (tokens < 0 || dim < 0) return record_error(MXFP4_ERR_INVALID_ARG, "%s: negative size", what);
    if (tokens > INT32_MAX || dim < 2 || dim > kMaxHeadDim || dim % 2)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: head_dim %lld must be even and at most %d, tokens below 2^31",
                            what, (long long)dim, kMaxHeadDim);
    if (!(eps >= 0.f)) return record_error(MXFP4_ERR_INVALID_ARG, "%s: eps must not be negative", what);
    p->tokens = (int32_t)tokens;
    p->dim = (int32_t)dim;
    p->eps = eps;
    p->pairs = 0;
    if (!rope) return MXFP4_OK;
    if (ids_dtype != MXFP4_IDS_I32 && ids_dtype != MXFP4_IDS_I64)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad ids_dtype %d", what, ids_dtype);
    if (rope->pairs < 0 || 2 * (int64_t)rope->pairs > dim)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: %d pairs do not fit head_dim %lld", what, rope->pairs,
                            (long long)dim);
    if (rope->interleaved != 0 && rope->interleaved != 1)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1", what);
    if (rope->pairs > 0 && (!rope->freq || axes < 1 || axes > 255))
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: freq is NULL or axes not in 1..255", what);
    if (rope->pairs > 0 && tokens > 0) {
        if (!positions) return record_error(MXFP4_ERR_INVALID_ARG, "%s: positions is NULL", what);
        if (reinterpret_cast<uintptr_t>(positions) % (ids_dtype == MXFP4_IDS_I64 ? 8 : 4))
            return record_error(MXFP4_ERR_MISALIGNED, "%s: positions not aligned to their type", what);
    }
    p->pairs = rope->pairs;
    p->interleaved = rope->interleaved;
    p->positions = positions;
    p->is64 = ids_dtype == MXFP4_IDS_I64;
    for (int i = 0; i < rope->pairs; ++i) {
        const double f = rope->freq[i];
        const int a = rope->axis ? rope->axis[i] : 0;
        if (!std::isfinite(f) || std::fabs(f) > 1e6)
            return record_error(MXFP4_ERR_INVALID_ARG, "%s: frequency %d is not finite or above 1e6", what, i);
        if (a < 0 || a >= axes)
            return record_error(MXFP4_ERR_INVALID_ARG, "%s: pair %d has axis %d of %lld", what, i, a, (long long)axes);
        p->freq[i] = fixed_turns(f);
        p->axis[i] = (uint8_t)a;
    }
    return MXFP4_OK;
}

mxfp4_status check_gain(const char* what, const char* name, const float* gain) {
    if (reinterpret_cast<uintptr_t>(gain) % 4)
        return record_error(MXFP4_ERR_MISALIGNED, "%s: %s not aligned to its element type", what, name);
    return MXFP4_OK;
}

RopeSide side_of(const Heads& x, const Heads& dy, const Heads& y, int32_t heads, const float* gain) {
    const int64_t size = heads_esize(y.dtype);
    return {x.data, dy.data, y.data, x.token_stride * size, x.head_stride * size, dy.token_stride * size,
            dy.head_stride * size, y.token_stride * size, y.head_stride * size, heads, gain};
}

// Pairs that a lane moves as runs of elements: the most that every row of every tensor allows.
int pairs_per_lane(const RopeParams& p, const Heads* const* all, int n) {
    const int half = p.dim / 2;
    for (int vec = 8; vec > 1; vec /= 2) {
        bool fits = half % vec == 0 && (p.interleaved || p.pairs % vec == 0);
        for (int i = 0; i < n && fits; ++i)
            if (all[i]->data) fits = heads_aligned(*all[i], vec * heads_esize(all[i]->dtype));
        if (fits) return vec;
    }
    return 1;
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" mxfp4_status mxfp4_qk_norm_rope(const mxfp4_heads* q, const mxfp4_heads* k, int64_t tokens, int64_t head_dim,
                                           const float* q_gain, const float* k_gain, float eps, const mxfp4_rope* rope,
                                           const void* positions, int ids_dtype, int64_t axes,
                                           const mxfp4_heads* q_out, const mxfp4_heads* k_out, mxfp4_stream_t stream) {
    const char* what = "qk_norm_rope";
    RopeParams p{};
    mxfp4_status st = rope_common(what, tokens, head_dim, eps, rope, positions, ids_dtype, axes, &p);
    if (st) return st;
    const mxfp4_heads* given[2][2] = {{q, q_out}, {k, k_out}};
    const float* gains[2] = {q_gain, k_gain};
    const char* names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    Heads h[2][2] = {};
    const Heads* all[4];
    for (int i = 0; i < 2; ++i) {
        if (i == 1 && !k) {  // queries alone
            all[2] = all[3] = &h[1][0];
            continue;
        }
        for (int j = 0; j < 2; ++j) {
            if ((st = check_heads(what, names[i][j], given[i][j], tokens, head_dim, j == 1, &h[i][j]))) return st;
            all[2 * i + j] = &h[i][j];
        }
        if (h[i][0].heads != h[i][1].heads || h[i][0].dtype != h[0][0].dtype || h[i][1].dtype != h[0][0].dtype)
            return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s has other heads or another type than %s or q", what,
                                names[i][1], names[i][0]);
        if ((st = check_gain(what, i ? "k_gain" : "q_gain", gains[i]))) return st;
        p.side[i] = side_of(h[i][0], Heads{}, h[i][1], h[i][0].heads, gains[i]);
    }
    if (tokens == 0) return record_error(MXFP4_OK, "%s", "");
    if ((st = ensure_device())) return st;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) {
        const int vec = pairs_per_lane(p, all, 4);
        int ctas = 0;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        e = launch_rope<false>(p, h[0][0].dtype, vec, sms, &ctas, s);
    }
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}

extern "C" size_t mxfp4_qk_norm_rope_grad_workspace_bytes(int64_t tokens, int64_t head_dim) {
    if (tokens <= 0 || tokens > INT32_MAX || head_dim < 2 || head_dim > kMaxHeadDim || head_dim % 2) return 0;
    return (size_t)kMaxCtas * 2 * (size_t)head_dim * sizeof(float);
}

extern "C" mxfp4_status mxfp4_qk_norm_rope_grad(const mxfp4_heads* q, const mxfp4_heads* k, const mxfp4_heads* dq,
                                                const mxfp4_heads* dk, int64_t tokens, int64_t head_dim,
                                                const float* q_gain, const float* k_gain, float eps,
                                                const mxfp4_rope* rope, const void* positions, int ids_dtype,
                                                int64_t axes, const mxfp4_heads* dq_in, const mxfp4_heads* dk_in,
                                                float* dq_gain, float* dk_gain, void* ws, size_t ws_bytes,
                                                mxfp4_stream_t stream) {
    const char* what = "qk_norm_rope_grad";
    RopeParams p{};
    mxfp4_status st = rope_common(what, tokens, head_dim, eps, rope, positions, ids_dtype, axes, &p);
    if (st) return st;
    const mxfp4_heads* given[2][3] = {{dq, dq_in, q}, {dk, dk_in, k}};
    const float* gains[2] = {q_gain, k_gain};
    float* dgains[2] = {dq_gain, dk_gain};
    const char* names[2][3] = {{"dq", "dq_in", "q"}, {"dk", "dk_in", "k"}};
    Heads h[2][3] = {};
    const Heads* all[6];
    bool sums = false;
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 3; ++j) all[3 * i + j] = &h[i][j];
        if (dgains[i] && (!gains[i] || !given[i][0]))
            return record_error(MXFP4_ERR_INVALID_ARG, "%s: a gradient of a gain that is not there", what);
        if (i == 1 && !dk) continue;  // queries alone
        for (int j = 0; j < (gains[i] ? 3 : 2); ++j) {  // without a norm x is not needed
            if ((st = check_heads(what, names[i][j], given[i][j], tokens, head_dim, j == 1, &h[i][j]))) return st;
            if (h[i][j].heads != h[i][0].heads || h[i][j].dtype != h[0][0].dtype)
                return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s has other heads or another type than %s or dq", what,
                                    names[i][j], names[i][0]);
        }
        if ((st = check_gain(what, i ? "k_gain" : "q_gain", gains[i]))) return st;
        if ((st = check_gain(what, i ? "dk_gain" : "dq_gain", dgains[i]))) return st;
        sums = sums || dgains[i];
        p.side[i] = side_of(h[i][2], h[i][0], h[i][1], h[i][0].heads, gains[i]);
    }
    if (sums && tokens > 0) {
        const size_t need = mxfp4_qk_norm_rope_grad_workspace_bytes(tokens, head_dim);
        if (!ws || ws_bytes < need)
            return record_error(MXFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", what, need);
        if (reinterpret_cast<uintptr_t>(ws) % 256)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: workspace not 256-byte aligned", what);
    }
    if (tokens == 0 && !sums) return record_error(MXFP4_OK, "%s", "");
    if ((st = ensure_device())) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (tokens == 0) {
        for (float* g : dgains)
            if (g && e == cudaSuccess) e = cudaMemsetAsync(g, 0, (size_t)head_dim * sizeof(float), s);
        if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s clear: %s", what, cudaGetErrorString(e));
        return record_error(MXFP4_OK, "%s", "");
    }
    int sms = 0;
    e = sm_count(&sms);
    if (e == cudaSuccess) {
        const int vec = pairs_per_lane(p, all, 6);
        int ctas = 0;
        p.partial = sums ? static_cast<float*>(ws) : nullptr;
        e = launch_rope<true>(p, h[0][0].dtype, vec, sms, &ctas, s);
        if (e == cudaSuccess && sums)
            e = launch_overlapped(rope_gain_kernel, dim3((unsigned)((head_dim + 31) / 32), 2), dim3(1024), 0, s, 1, true,
                                  (const float*)p.partial, ctas, (int)head_dim, dq_gain, dk_gain);
    }
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}
