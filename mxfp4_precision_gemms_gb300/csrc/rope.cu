// rope.cu -- norm of each head of queries and keys with the rotation by position in the same pass, and its gradient.
//
//   r = 1 / sqrt(mean x^2 + eps),  n = x r gain          (no gain: n = x)
//   (a, b) -> (a cos - b sin, b cos + a sin),  angle = positions[axis of the pair][token] * freq[pair]
// Backwards, with dz the gradient turned back by the same angles and u = x r:
//   dx = r (dz gain - u mean(dz gain u)),   dgain = sum over tokens and heads of dz u
//
// HBM bandwidth bounds long calls, latency short ones.  A CTA takes a few tokens: first it makes the cosines and sines
// of each token and pair in shared memory, once for all heads, then groups of lanes take the rows (a token's head).  A
// lane holds VEC pairs, as two runs of VEC elements (or one of 2 VEC, where a pair's elements are neighbours), and every
// row is read once and written once.  The elements behind the rotated ones are pairs that do not turn.
//
// Angles.  A position times a frequency in fp32 is off by 2^-24 of itself, which is 0.03 radians at position 500000.  Here a
// frequency is held as turns per position in 64-bit fixed point, and a product with an integer modulo 2^64 is the exact
// fraction of a turn: what is left is the frequency's own rounding (2^-65 turns a position), whatever the position.
#include <algorithm>
#include <cmath>

#include "element.cuh"
#include "heads.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kRopeThreads = 256;
constexpr int kMaxHeadDim = 256;
constexpr int kMaxPairs = kMaxHeadDim / 2;
constexpr int kTokens = 8;      // tokens of a CTA's turn
constexpr int kCtasPerSm = 4;   // partial sums of the gains' gradients: one row for each CTA

struct RopeSide {  // queries or keys
    const void* x;
    const void* dy;  // gradient only
    void* y;         // the result: y, or dx
    int64_t x_token, x_head, dy_token, dy_head, y_token, y_head;
    int32_t heads;
    const float* gain;
};

struct RopeParams {
    RopeSide side[2];
    int32_t tokens, dim, pairs, interleaved, is64, per_turn;
    float eps;
    const void* positions;  // [axes][tokens]
    float* partial;         // gradient only: [CTA][2][dim]
    uint64_t freq[kMaxPairs];
    uint8_t axis[kMaxPairs];
};

// VEC neighbouring elements, aligned to their size in bytes (at most 32).
template <int VEC, class T>
__device__ __forceinline__ void load_run(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 8)
        unpack8(load8(p), v);
    else if constexpr (VEC == 4)
        load4(p, v);
    else
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = load1(p + i);
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

// The pairs [at, at + VEC) of a row: a[i], b[i].
template <int VEC, class T>
__device__ __forceinline__ void load_pairs(const T* row, int at_a, int at_b, int interleaved, float (&a)[VEC],
                                           float (&b)[VEC]) {
    float u[VEC], v[VEC];
    load_run<VEC>(row + at_a, u);
    load_run<VEC>(row + at_b, v);
    if (interleaved && VEC > 1) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            a[i] = 2 * i < VEC ? u[(2 * i) % VEC] : v[(2 * i) % VEC];
            b[i] = 2 * i + 1 < VEC ? u[(2 * i + 1) % VEC] : v[(2 * i + 1) % VEC];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[i] = u[i], b[i] = v[i];
    }
}
template <int VEC, class T>
__device__ __forceinline__ void store_pairs(T* row, int at_a, int at_b, int interleaved, const float (&a)[VEC],
                                            const float (&b)[VEC]) {
    float u[VEC], v[VEC];
    if (interleaved && VEC > 1) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            u[i] = i % 2 ? b[i / 2] : a[i / 2];
            v[i] = i % 2 ? b[(VEC + i) / 2] : a[(VEC + i) / 2];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) u[i] = a[i], v[i] = b[i];
    }
    store_run<VEC>(row + at_a, u);
    store_run<VEC>(row + at_b, v);
}

// Sum over the `n` lanes of a row's group, in every one of them (li: this lane's place in it).
__device__ __forceinline__ float group_sum(float v, int li, int n) {
    const int lane = threadIdx.x & 31;
    for (int o = n <= 1 ? 0 : 1 << (31 - __clz(n - 1)); o > 0; o >>= 1) {
        const float t = __shfl_down_sync(0xffffffffu, v, o);
        if (li < o && li + o < n) v += t;
    }
    return __shfl_sync(0xffffffffu, v, lane - li);
}

// SLOTS: runs of pairs of a lane, 32 lanes apart (rows of more than 32 VEC pairs).
template <class T, int VEC, int SLOTS, bool GRAD>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 turn[kTokens * kMaxPairs];
    grid_dependency_wait();
    allow_dependent_launch();
    const int half = p.dim / 2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = min(32, half / VEC);  // of a row
    const int per_warp = 32 / lanes;        // rows that a warp takes at once
    const int li = lane % lanes, sub = lane / lanes;
    const bool idle = sub >= per_warp;
    const int groups = kRopeThreads / 32 * per_warp, group = warp * per_warp + sub;
    // where this lane's elements are
    int at_a[SLOTS], at_b[SLOTS], pair[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int c = (li + s * lanes) * VEC;  // first pair
        pair[s] = c < half ? c : -1;
        if (p.interleaved) {
            at_a[s] = 2 * c, at_b[s] = 2 * c + VEC;
        } else if (c < p.pairs) {
            at_a[s] = c, at_b[s] = c + p.pairs;
        } else {
            at_a[s] = p.pairs + c, at_b[s] = half + c;
        }
    }

    float dgain[GRAD ? 2 : 1][SLOTS][2][VEC] = {};
    const int turns = (p.tokens + p.per_turn - 1) / p.per_turn;
    for (int it = blockIdx.x; it < turns; it += gridDim.x) {
        const int t0 = it * p.per_turn, nt = min(p.per_turn, p.tokens - t0);
        __syncthreads();  // the cosines of the turn before have been read
        for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
            const int t = i / half, c = i - t * half;
            float2 cs = make_float2(1.f, 0.f);
            if (c < p.pairs) {
                const int64_t pos = load_id(p.positions, p.is64, (int64_t)p.axis[c] * p.tokens + t0 + t);
                const int64_t frac = (int64_t)((uint64_t)pos * p.freq[c]);  // of a turn, times 2^64
                sincospif((float)frac * 0x1p-63f, &cs.y, &cs.x);
            }
            turn[i] = cs;
        }
        __syncthreads();
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const RopeSide& side = p.side[which];
            const int rows = nt * side.heads;
            float gain[SLOTS][2][VEC];
            if (side.gain) {
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (pair[s] >= 0) {
                        float u[VEC], v[VEC];
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            u[i] = __ldg(side.gain + at_a[s] + (p.interleaved ? 2 * i : i));
                            v[i] = __ldg(side.gain + (p.interleaved ? at_a[s] + 2 * i + 1 : at_b[s] + i));
                        }
#pragma unroll
                        for (int i = 0; i < VEC; ++i) gain[s][0][i] = u[i], gain[s][1][i] = v[i];
                    }
            }
            // whole warps go round together: the sums are over lanes
            for (int r0 = warp * per_warp; r0 < rows; r0 += groups) {
                const int r = r0 + sub;
                const bool on = !idle && r < rows;
                const int t = on ? r / side.heads : 0, h = on ? r - t * side.heads : 0;
                const int64_t token = t0 + t;
                const T* x = static_cast<const T*>(side.x) + token * side.x_token + h * side.x_head;
                T* y = static_cast<T*>(side.y) + token * side.y_token + h * side.y_head;
                const float2* cs = turn + t * half;
                float a[SLOTS][VEC] = {}, b[SLOTS][VEC] = {};
                float da[SLOTS][VEC] = {}, db[SLOTS][VEC] = {};
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (on && pair[s] >= 0) {
                        if (!GRAD || side.gain) load_pairs<VEC>(x, at_a[s], at_b[s], p.interleaved, a[s], b[s]);
                        if constexpr (GRAD) {
                            const T* dy = static_cast<const T*>(side.dy) + token * side.dy_token + h * side.dy_head;
                            load_pairs<VEC>(dy, at_a[s], at_b[s], p.interleaved, da[s], db[s]);
                        }
                    }
                if (side.gain) {
                    float ss = 0.f;
#pragma unroll
                    for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) ss = fmaf(a[s][i], a[s][i], fmaf(b[s][i], b[s][i], ss));
                    const float rstd = rsqrtf(group_sum(ss, li, lanes) / (float)p.dim + p.eps);
#pragma unroll
                    for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) a[s][i] *= rstd, b[s][i] *= rstd;
                    if constexpr (GRAD) {
                        float dot = 0.f;
#pragma unroll
                        for (int s = 0; s < SLOTS; ++s)
                            if (on && pair[s] >= 0) {
#pragma unroll
                                for (int i = 0; i < VEC; ++i) {
                                    const float2 c = cs[pair[s] + i];
                                    const float za = fmaf(da[s][i], c.x, db[s][i] * c.y);
                                    const float zb = fmaf(db[s][i], c.x, -da[s][i] * c.y);
                                    dgain[which][s][0][i] = fmaf(za, a[s][i], dgain[which][s][0][i]);
                                    dgain[which][s][1][i] = fmaf(zb, b[s][i], dgain[which][s][1][i]);
                                    da[s][i] = za * gain[s][0][i], db[s][i] = zb * gain[s][1][i];
                                    dot = fmaf(da[s][i], a[s][i], fmaf(db[s][i], b[s][i], dot));
                                }
                            }
                        dot = group_sum(dot, li, lanes) / (float)p.dim;
#pragma unroll
                        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) {
                                a[s][i] = (da[s][i] - a[s][i] * dot) * rstd;
                                b[s][i] = (db[s][i] - b[s][i] * dot) * rstd;
                            }
                    }
                }
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (on && pair[s] >= 0) {
                        if constexpr (!GRAD) {
#pragma unroll
                            for (int i = 0; i < VEC; ++i) {
                                const float2 c = cs[pair[s] + i];
                                const float u = side.gain ? a[s][i] * gain[s][0][i] : a[s][i];
                                const float v = side.gain ? b[s][i] * gain[s][1][i] : b[s][i];
                                a[s][i] = fmaf(u, c.x, -v * c.y), b[s][i] = fmaf(v, c.x, u * c.y);
                            }
                        } else if (!side.gain) {
#pragma unroll
                            for (int i = 0; i < VEC; ++i) {
                                const float2 c = cs[pair[s] + i];
                                a[s][i] = fmaf(da[s][i], c.x, db[s][i] * c.y);
                                b[s][i] = fmaf(db[s][i], c.x, -da[s][i] * c.y);
                            }
                        }
                        store_pairs<VEC>(y, at_a[s], at_b[s], p.interleaved, a[s], b[s]);
                    }
            }
        }
    }
    if constexpr (GRAD) {
        if (!p.partial) return;
        // the groups' sums, added up in their order
        __shared__ float sums[kRopeThreads / 32 * 32 * VEC * 2 * SLOTS];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            if (!idle) {
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (pair[s] >= 0) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            float* to = sums + group * p.dim;
                            to[at_a[s] + (p.interleaved ? 2 * i : i)] = dgain[which][s][0][i];
                            to[p.interleaved ? at_a[s] + 2 * i + 1 : at_b[s] + i] = dgain[which][s][1][i];
                        }
                    }
            }
            __syncthreads();
            for (int d = threadIdx.x; d < p.dim; d += kRopeThreads) {
                float v = 0.f;
                for (int g = 0; g < groups; ++g) v += sums[g * p.dim + d];
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

constexpr int kMaxCtas = 148 * 8;  // bounds the workspace; more SMs than that need no more

// CTAs of a call, and how many tokens each takes at a time: as many CTAs as there are turns of kTokens, no fewer than
// SMs, no more than fit the device at once; then the tokens shared out so that all take as many turns.
int rope_ctas(int64_t tokens, int sms, int32_t* per_turn) {
    const int64_t most = std::min<int64_t>(kMaxCtas, (int64_t)sms * kCtasPerSm);
    const int64_t turns = (tokens + kTokens - 1) / kTokens;
    const int64_t ctas = std::min(std::max(turns, std::min<int64_t>(tokens, sms)), most);
    const int64_t rounds = (tokens + ctas * kTokens - 1) / (ctas * kTokens);
    *per_turn = (int32_t)((tokens + ctas * rounds - 1) / (ctas * rounds));
    return (int)ctas;
}

template <class T, bool GRAD>
cudaError_t launch_rope(const RopeParams& p, int vec, int ctas, cudaStream_t s) {
    const dim3 grid((unsigned)ctas), block(kRopeThreads);
    if (vec == 8) return launch_overlapped(rope_kernel<T, 8, 1, GRAD>, grid, block, 0, s, 1, true, p);
    if (vec == 4) return launch_overlapped(rope_kernel<T, 4, 1, GRAD>, grid, block, 0, s, 1, true, p);
    if (vec == 2) return launch_overlapped(rope_kernel<T, 2, 2, GRAD>, grid, block, 0, s, 1, true, p);
    return launch_overlapped(rope_kernel<T, 1, 4, GRAD>, grid, block, 0, s, 1, true, p);
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
        p.side[i] = {h[i][0].data, nullptr, h[i][1].data, h[i][0].token_stride, h[i][0].head_stride, 0, 0,
                     h[i][1].token_stride, h[i][1].head_stride, h[i][0].heads, gains[i]};
    }
    if (tokens == 0) return record_error(MXFP4_OK, "%s", "");
    if ((st = ensure_device())) return st;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) {
        const int vec = pairs_per_lane(p, all, 4), ctas = rope_ctas(tokens, sms, &p.per_turn);
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        e = h[0][0].dtype == MXFP4_OUT_BF16 ? launch_rope<bf16, false>(p, vec, ctas, s)
                                            : launch_rope<float, false>(p, vec, ctas, s);
    }
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}

extern "C" size_t mxfp4_qk_norm_rope_grad_workspace_bytes(int64_t tokens, int64_t head_dim) {
    if (tokens <= 0 || tokens > INT32_MAX || head_dim < 2 || head_dim > kMaxHeadDim || head_dim % 2) return 0;
    return (size_t)std::min<int64_t>(kMaxCtas, tokens) * 2 * (size_t)head_dim * sizeof(float);
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
        p.side[i] = {h[i][2].data, h[i][0].data, h[i][1].data, h[i][2].token_stride, h[i][2].head_stride,
                     h[i][0].token_stride, h[i][0].head_stride, h[i][1].token_stride, h[i][1].head_stride, h[i][0].heads,
                     gains[i]};
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
        const int vec = pairs_per_lane(p, all, 6), ctas = rope_ctas(tokens, sms, &p.per_turn);
        p.partial = sums ? static_cast<float*>(ws) : nullptr;
        e = h[0][0].dtype == MXFP4_OUT_BF16 ? launch_rope<bf16, true>(p, vec, ctas, s)
                                            : launch_rope<float, true>(p, vec, ctas, s);
        if (e == cudaSuccess && sums)
            e = launch_overlapped(rope_gain_kernel, dim3((unsigned)((head_dim + 31) / 32), 2), dim3(1024), 0, s, 1, true,
                                  (const float*)p.partial, ctas, (int)head_dim, dq_gain, dk_gain);
    }
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}
