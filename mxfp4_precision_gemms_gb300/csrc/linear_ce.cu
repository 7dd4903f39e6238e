// linear_ce.cu -- softmax cross entropy of a linear output layer, without its logits in memory,
// and its gradients.
//
//   z = h w^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_{t, y_t}
//   dz_tv = g_t (exp(z_tv - lse_t) - [v = y_t]),  dh = dz w,  dw = dz^T h
//
// Everything of size tokens x vocab lives in tensor memory and registers, except one piece of dz
// (all tokens x a range of the vocabulary, bf16) between the kernel that makes it and the one
// that multiplies it.  The forward pass is one matrix product (2 T V D operations), the backward
// pass three: the logits are made again (the price of not keeping them), and two gradients.
// All of them are compute-bound for T above a few hundred tokens; for few tokens the read of w (and
// the write of dw) from HBM bounds them.
//
//   gather    copies the counted rows of h together: ignored rows cost no multiplication, and what they
//             hold cannot reach a sum (left out before the loss of at most 256 tokens)
//   stats     logits tile by tile; each thread reduces 128 columns of one row to (max, sum)
//   combine   joins the tiles' statistics, writes lse and the losses
//   dlogits   logits of one piece again -> dz in bf16 (as the sum of two for at most 128 tokens)
//   products  dh += dz w and dw = dz^T h of that piece, in one launch
//   scatter   adds up the parts of dh and puts its rows back in the tokens' order
//
// The three matrix kernels share one structure, a persistent kernel of CTA pairs with 256 x 256
// tiles (tcgen05.mma.cta_group::2.kind::f16, K = 64 per stage):
//   warp 0     TMA producer of this CTA's 128 rows of A and 128 of B, six stages deep
//   warp 1     allocates TMEM; in the even CTA one thread issues the pair's MMAs
//   warps 2-9  epilogue of this CTA's 128 rows, two warps per lane quadrant
// Two accumulators (all 512 columns of TMEM): an epilogue overlaps the next tile's MMAs.
// Operands lie in shared memory as the tensors lie in HBM, with 128-byte rows along K (h, w, and dz
// as rows of tokens) or along M / N (w and h as summands, dz for dw): nothing is transposed.
#include <algorithm>

#include "element.cuh"
#include "step_ops.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kTile = 256;    // rows and columns of a pair's tile
constexpr int kK = 64;        // K per stage: 128 bytes of bf16
constexpr int kStages = 6;
constexpr int kOpBytes = 128 * kK * 2;  // one CTA's half of an operand's stage
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBoxBytes = 32 * 64;  // staging box of a TMA store: 32 rows x 64 bytes, 64-byte swizzle
constexpr int kBoxes = 2;           // per epilogue warp
constexpr int kOffA = 0;
constexpr int kOffB = kOffA + kStages * kOpBytes;
constexpr int kOffBox = kOffB + kStages * kOpBytes;
constexpr int kOffBar = kOffBox + kEpiWarps * kBoxes * kBoxBytes;
constexpr int kNumBars = 2 * kStages + 5;
constexpr int kOffTmem = kOffBar + kNumBars * 8;
constexpr int kSmem = kOffTmem + 16;
static_assert(kSmem <= 227 * 1024, "shared memory budget");
static_assert(2 * kSmem > 228 * 1024, "one CTA per SM: two pairs never compete for TMEM");
static_assert(kOffBox % 1024 == 0 && kOffBar % 8 == 0, "alignment");

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What the gather kernel leaves for the others.  The forward pass of at most one tile of tokens has
// none: its rows are read where they lie (a row's values reach no other row's logits).
struct Header {
    int32_t count;  // tokens that count
    float gscale;   // factor that every token's gradient shares
};

// Read as volatile, by value: as an lvalue next to a kernel parameter in a conditional expression it
// would make the parameter's own read volatile too, which parameter memory does not take (a fault).
__device__ __forceinline__ int32_t counted_tokens(const Header* h) {
    return *reinterpret_cast<const volatile int32_t*>(&h->count);
}
__device__ __forceinline__ float shared_factor(const Header* h) {
    return *reinterpret_cast<const volatile float*>(&h->gscale);
}

// One matrix product C[M, N] (+)= A[M, K] . B[N, K]^T, or a launch's share of two.
struct Product {
    CUtensorMap map_a, map_b, map_c;
    int32_t a_mn, b_mn;     // the operand's rows in memory run over K, its M / N index is contiguous
    int32_t m_counted;      // M is the number of counted tokens (rounded up to a tile)
    int32_t k_counted;      // K is the number of counted tokens
    int32_t M, N, K;
    int32_t tile_n;         // columns of a tile: kTile, or less where that divides better (a multiple of 32)
    int32_t num_n;          // tiles along N
    uint32_t tx;            // bytes of a stage, both CTAs
    int32_t splits;         // K is cut into this many parts, each with its own output
    int32_t k_per_split;    // stages of a part
    int32_t slot_rows;      // rows of C between the parts' outputs
    int32_t out_bf16, add;  // output type; add to what is there (fp32)
    int32_t scaled;         // multiply by Header::gscale
};

struct CeParams {
    Product prod[2];
    int32_t count;
    const Header* header;
    const int32_t* target;  // [rows] targets of the counted tokens
    // forward pass without a gather: all tokens are rows, their targets as the caller has them
    int32_t direct, tokens, is64;
    const void* targets;
    int32_t col0;           // first vocabulary index of this launch's columns
    int32_t rows;           // pitch of the statistics: padded token count
    int32_t paired;         // gradient of at most kPaired tokens: see there
    float2* stats;          // [tile * 2 + half][rows]: (max, sum of exp(z - max))
    float* target_logit;    // [rows]
    const float* lse2;      // [rows] lse * log2 e
    const float* ratio;     // [rows] factor of this token's gradient
    uint32_t* status;
    uint64_t wait_ns;
};

// dz is rounded to bf16 for the tensor cores, whatever the outputs' type (a second bf16 number for what
// rounding leaves would make both products twice as long).  Of 459 counted tokens of a 50021 x 1032 layer that leaves
// a bf16 dh off by 1.80e-3 of itself, where its own rounding is 1.66e-3.  Over many tokens the errors of their
// dz average out, over a few they need not (dz is largest at the target, and its error there goes into the
// whole row of dh).  At most kPaired tokens fill half
// of a tile's rows, so the other half, idle otherwise, holds their rows again with what the
// rounding left of dz: both products then sum dz to 16 bits, at no cost.  (dz itself is as exact as lse in
// fp32 lets p = exp(z - lse) be: 2^-23 |lse| of p, which a confident token's p - 1 feels.)
constexpr int32_t kPaired = 128;

enum Kind { kStats = 0, kDlogits = 1, kProducts = 2, kDlogitsFew = 3 };  // kDlogitsFew: paired

// Stages that one accumulator takes.  The tensor cores cut each step's sum off towards zero, and the
// loss of a long contraction would carry that one-sided error: the logits of dim = 4096 came out
// smaller by 4.2e-6 of themselves (1.0e-6 at 1024), ten times an fp32 product's error.  So the
// logits are summed in runs of K = 512, joined in fp32 by the epilogue, which has the time:
// a run is 4096 cycles of MMAs and about 500 of read-out.  Runs of 256 halve what error is left (4.5e-7 of a
// logit) and cost 3 to 6%; they are taken for at most a tile of tokens, where HBM is waited for anyway and
// few losses average an error out.  The gradients make the logits again in the same runs, so that z - lse
// has only lse's rounding: in one run z would be short of the lse that it is subtracted from, and
// p - 1 at the target of a confident token (logit 30) off by 1.3e-4 whatever it is.  (That costs the gradients
// of 8192 tokens 2 to 3% at dim = 640, 1% at 1024 and nothing that shows from 2048 on.)  The two gradient
// products have no such difference to keep, and are taken in one run.
constexpr int kLogitsRun = 8, kLogitsRunFew = 4;

__host__ __device__ inline int32_t pad_rows(int32_t n) { return n <= 0 ? kTile : (n + kTile - 1) / kTile * kTile; }

struct Tile {
    int prob;
    int32_t m0, n0, n_tile, k0, stages, slot;
};

// A tile's columns for N columns in all: as few tiles as 256-column ones, cut evenly.  The MMA's time
// goes with the columns (dim = 1032: five tiles of 224 instead of 256, an eighth less).
inline int32_t even_tile(int64_t n) {
    const int64_t tiles = (n + kTile - 1) / kTile;
    return (int32_t)(((n + tiles - 1) / tiles + 31) / 32 * 32);
}

inline uint32_t stage_bytes(int32_t b_columns) { return 2u * (128u + (uint32_t)b_columns / 2) * kK * 2; }

constexpr int kClustersMost = 76;  // pairs of SMs

// A tile's columns of the vocabulary where the tiles fill the device few times over: the width whose
// schedule is shortest.  A stage costs two cycles a column, or its bytes at 72 a cycle (what L2
// gives an SM), and a tile some 600 cycles more.  (64 tokens, 65536 x 2048: 256 tiles of 256 columns are
// four rounds of 76, and so are 293 of 224: 65 -> 61 us.)
inline int32_t vocab_tile(int64_t num_m, int64_t n, int64_t k) {
    if (num_m * ((n + kTile - 1) / kTile) >= 8 * kClustersMost) return kTile;
    int32_t best = kTile;
    int64_t best_cost = INT64_MAX;
    for (int32_t w = kTile; w >= 128; w -= 32) {
        const int64_t rounds = (num_m * ((n + w - 1) / w) + kClustersMost - 1) / kClustersMost;
        const int64_t stage = std::max<int64_t>(2 * w, stage_bytes(w) / 2 / 72);
        const int64_t cost = rounds * (stage * ((k + kK - 1) / kK) + 600);
        if (cost < best_cost) best = w, best_cost = cost;
    }
    return best;
}

__device__ __forceinline__ int32_t tiles_m(const Product& q, int32_t count) {
    return (q.m_counted ? pad_rows(count) : q.M + kTile - 1) / kTile;
}

// Tile `lt` of product `i`.  Consecutive tiles (which run at the same time) walk the dimension with
// fewer tiles first: the operand along it is read in every wave and stays in L2 while the other
// one streams through once.
__device__ __forceinline__ void locate(const CeParams& p, int32_t count, int i, int32_t lt, Tile& out) {
    const Product& q = p.prod[i];
    const int32_t num_m = tiles_m(q, count), num_n = q.num_n;
    out.prob = i;
    out.slot = 0;
    if (q.splits > 1) {
        out.slot = lt / (num_m * num_n);
        lt -= out.slot * (num_m * num_n);
    }
    // one division: it stands before a cluster's first load
    const int32_t inner = min(num_m, num_n), major = inner > 1 ? lt / inner : lt, minor = lt - major * inner;
    out.m0 = (num_n > num_m ? minor : major) * kTile;
    out.n_tile = num_n > num_m ? major : minor;
    out.n0 = out.n_tile * q.tile_n;
    const int32_t k = q.k_counted ? max(count, 1) : q.K;
    const int32_t all = (k + kK - 1) / kK;
    out.k0 = out.slot * q.k_per_split;
    out.stages = q.splits > 1 ? min(q.k_per_split, all - out.k0) : all;
}
__device__ __forceinline__ int32_t tiles_in(const CeParams& p, int32_t count, int i) {
    return tiles_m(p.prod[i], count) * p.prod[i].num_n * p.prod[i].splits;
}

// The tiles of one cluster, in order; every role of both CTAs walks the same ones.  One product:
// every num_clusters-th tile.  Two: the first one's tiles (the longer contraction) that way, and
// while `rest` clusters have one of them more than the others, those others take `lead` rounds of the
// second one's tiles; then all clusters take turns again.
template <int KIND>
struct Walk {
    int32_t cluster, clusters, tiles0, tiles1, rest, lead, turn;
    __device__ __forceinline__ void start(const CeParams& p, int32_t count, int32_t c, int32_t n) {
        cluster = c, clusters = n, turn = 0;
        tiles0 = tiles_in(p, count, 0);
        tiles1 = rest = lead = 0;
        if (KIND == kProducts && p.count == 2) {
            tiles1 = tiles_in(p, count, 1);
            rest = tiles0 % n;
            // A tile's time in stages: its own and two of hand-off, but no less than storing it takes
            // (128 KB at a pair's share of HBM: six stages, twelve for fp32).
            const Product& q = p.prod[1];
            const int32_t k = q.k_counted ? max(count, 1) : q.K;
            const int32_t one = max((k + kK - 1) / kK, q.out_bf16 ? 6 : 12) + 2;
            if (rest) lead = (p.prod[0].k_per_split + 2 + one / 2) / one;
        }
    }
    __device__ __forceinline__ bool next(const CeParams& p, int32_t count, Tile& t) {
        const int32_t j = turn++;
        const int32_t at = cluster + j * clusters;
        if (at < tiles0) {
            locate(p, count, 0, at, t);
            return true;
        }
        if (KIND != kProducts || tiles1 == 0) return false;
        const int32_t i = j - (tiles0 / clusters + (cluster < rest ? 1 : 0));
        const int32_t ahead = clusters - rest;  // clusters that take the lead rounds
        int32_t lt;
        if (cluster < rest)
            lt = lead * ahead + i * clusters + cluster;
        else if (i < lead)
            lt = i * ahead + cluster - rest;
        else
            lt = lead * ahead + (i - lead) * clusters + cluster;
        if (lt >= tiles1) return false;
        locate(p, count, 1, lt, t);
        return true;
    }
};

// Lane i writes its row's 64 bytes into a staging box (16-byte piece j of row r at
// j ^ ((r >> 1) & 3): the 64-byte swizzle, conflict-free).
__device__ __forceinline__ void write_box(uint8_t* box, int lane, const uint32_t* w) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// A warp's staging boxes, used in turn: a box is written again once the store before the last
// has read it.
struct Boxes {
    uint8_t* base;
    int turn;
    __device__ __forceinline__ void store(const CUtensorMap* map, int lane, const uint32_t* w, int32_t x, int32_t y,
                                          bool inside, bool add) {
        if (lane == 0) bulk_wait_read<kBoxes - 1>();
        __syncwarp();
        uint8_t* box = base + turn * kBoxBytes;
        turn = turn + 1 == kBoxes ? 0 : turn + 1;
        write_box(box, lane, w);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (inside) {
                if (add)
                    tma_reduce_add_2d(map, box, x, y);
                else
                    tma_store_2d(map, box, x, y);
            }
            bulk_commit();
        }
    }
};

// Compute-bound for many tokens: 2048 x 65536 x 4096, statistics 0.55 ms, dz 0.57 ms, both products 1.13 ms, with
// the tensor pipe active in 98.8, 96.4 and 96.7% of the cycles at the 1.68 to 1.71 GHz that the power cap leaves
// (1.9 to 2.0 PFLOP/s; a cuBLAS product of 8192^3 reached 1.89).
template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) ce_matrix_kernel(const __grid_constant__ CeParams p) {
    extern __shared__ uint8_t smem[];
    // The swizzled tiles need 1024-byte alignment.  Both CTAs of a pair see the same base, so
    // both return here, before any cluster barrier.
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusSmemLayout);
        return;
    }
    uint8_t* sA = smem + kOffA;
    uint8_t* sB = smem + kOffB;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);  // used in the leader
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;   // [2]
    uint64_t* acc_empty = acc_full + 2;     // [2], used in the leader: both CTAs' epilogues arrive
    uint64_t* mma_done = acc_empty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffTmem);

    // stages per accumulator, a power of two
    const int32_t run = KIND == kProducts ? 1 << 30 : p.rows <= kTile ? kLogitsRunFew : kLogitsRun;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int32_t cluster = (int32_t)(blockIdx.x >> 1), num_clusters = (int32_t)(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 2 * kEpiWarps);
        }
        mbar_init(mma_done, 1);
        fence_mbar_init();
        for (int i = 0; i < p.count; ++i) {
            prefetch_tmap(&p.prod[i].map_a);
            prefetch_tmap(&p.prod[i].map_b);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other's
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // The set-up above touches no global memory, so it overlaps the previous kernel.
    grid_dependency_wait();
    allow_dependent_launch();
    int32_t count = p.tokens;
    if (KIND != kStats || !p.direct) count = counted_tokens(p.header);
    const int32_t rows = KIND != kStats && p.paired ? kTile : count;  // that hold something

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs)
        if (elect_one()) {
            const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
            uint32_t armed[kStages];  // phases issued per stage
#pragma unroll
            for (int s = 0; s < kStages; ++s) armed[s] = 0;
            uint32_t s = 0, round = 0;
            bool ok = true;
            Tile t;
            Walk<KIND> walk;
            walk.start(p, rows, cluster, num_clusters);
            while (ok && walk.next(p, rows, t)) {
                const Product& q = p.prod[KIND == kProducts ? t.prob : 0];
                const int32_t ya = t.m0 + (int32_t)rank * 128, yb = t.n0 + (int32_t)rank * (q.tile_n / 2);
                for (int32_t i = 0; i < t.stages; ++i) {
                    if (round > 0 && !wait_bounded(&empty[s], (round - 1) & 1u, p.wait_ns, p.status)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], q.tx);
                    const uint32_t bar = full_leader + s * 8u;
                    const int32_t k = (t.k0 + i) * kK;
                    uint8_t* a = sA + s * kOpBytes;
                    uint8_t* b = sB + s * kOpBytes;
                    if (q.a_mn) {  // two boxes of 64 rows (K) x 64 columns (M)
                        tma_load_2d_pair(a, &q.map_a, bar, ya, k);
                        tma_load_2d_pair(a + kOpBytes / 2, &q.map_a, bar, ya + 64, k);
                    } else {  // one box of 128 rows (M) x 64 columns (K)
                        tma_load_2d_pair(a, &q.map_a, bar, k, ya);
                    }
                    if (q.b_mn) {
                        tma_load_2d_pair(b, &q.map_b, bar, yb, k);
                        tma_load_2d_pair(b + kOpBytes / 2, &q.map_b, bar, yb + 64, k);
                    } else {
                        tma_load_2d_pair(b, &q.map_b, bar, k, yb);
                    }
#pragma unroll
                    for (int j = 0; j < kStages; ++j)
                        if (j == (int)s) armed[j] = round + 1;
                    if (++s == kStages) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // Drain: the leader waits until the last armed phase of every stage has landed, both
            // CTAs until the MMAs have released every stage they were given.
#pragma unroll
            for (int j = 0; j < kStages; ++j) {
                if (!armed[j]) continue;
                if (rank == 0) wait_bounded(&full[j], (armed[j] - 1u) & 1u, p.wait_ns, p.status);
                wait_bounded(&empty[j], (armed[j] - 1u) & 1u, p.wait_ns, p.status);
            }
        }
    } else if (warp == 1) {
        // ---------------- tensor-core issuer (leader CTA)
        if (elect_one()) {
            if (rank == 0) {
                uint32_t s = 0, phase = 0, tcount = 0;
                bool ok = true;
                Tile t;
                Walk<KIND> walk;
                walk.start(p, rows, cluster, num_clusters);
                while (ok && walk.next(p, rows, t)) {
                    const Product& q = p.prod[KIND == kProducts ? t.prob : 0];
                    const uint32_t idesc = idesc_bf16(256, (uint32_t)q.tile_n, q.a_mn != 0, q.b_mn != 0);
                    // K = 16 further on: 32 bytes along a K-contiguous row, 16 rows of 128 bytes otherwise.
                    // Between 64-column blocks of M / N: half a stage's operand.
                    const uint32_t a_step = q.a_mn ? 2048 : 32, b_step = q.b_mn ? 2048 : 32;
                    const uint32_t a_lbo = q.a_mn ? kOpBytes / 2 : 16, b_lbo = q.b_mn ? kOpBytes / 2 : 16;
                    uint32_t d = 0;
                    for (int32_t i = 0; i < t.stages; ++i) {
                        const bool first = (i & (run - 1)) == 0;
                        if (first) {  // a new accumulator
                            const uint32_t ab = tcount & 1u;
                            if (tcount >= 2 &&
                                !wait_bounded(&acc_empty[ab], ((tcount >> 1) - 1u) & 1u, p.wait_ns, p.status)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            d = tmem + ab * 256;
                        }
                        if (!wait_bounded(&full[s], phase, p.wait_ns, p.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a = smem_u32(sA + s * kOpBytes), b = smem_u32(sB + s * kOpBytes);
#pragma unroll
                        for (int k = 0; k < kK / 16; ++k)
                            tc_mma_bf16_pair(d, smem_desc(a + k * a_step, a_lbo, 1024, kSwizzle128B),
                                             smem_desc(b + k * b_step, b_lbo, 1024, kSwizzle128B), idesc,
                                             !first || k != 0);
                        tc_commit_pair(&empty[s], 0x3);
                        if (++s == kStages) {
                            s = 0;
                            phase ^= 1u;
                        }
                        if ((i & (run - 1)) == run - 1 || i + 1 == t.stages) {
                            tc_commit_pair(&acc_full[tcount & 1u], 0x3);
                            ++tcount;
                        }
                    }
                }
                tc_commit_pair(mma_done, 0x3);
            }
            // Both CTAs: every MMA of the pair has completed before TMEM is released.
            wait_bounded(mma_done, 0, p.wait_ns, p.status);
        }
    } else {
        // ---------------- epilogue (both CTAs): this CTA's 128 rows of the tile
        const int quad = warp & 3;
        const int half = (warp - 2) >> 2;
        Boxes boxes{smem + kOffBox + (warp - 2) * kBoxes * kBoxBytes, 0};
        const uint32_t acc_empty_leader = mapa_shared(smem_u32(acc_empty), 0);
        float gscale = 1.f;
        if constexpr (KIND == kProducts) gscale = shared_factor(p.header);
        uint32_t tcount = 0;
        bool ok = true;
        Tile t;
        Walk<KIND> walk;
        walk.start(p, rows, cluster, num_clusters);
        while (ok && walk.next(p, rows, t)) {
            const Product& q = p.prod[KIND == kProducts ? t.prob : 0];
            const int32_t row0 = t.m0 + (int32_t)rank * 128 + quad * 32;
            const int32_t row = row0 + lane;
            const int32_t c0 = t.n0 + half * 128;
            // per-row values first: their latency hides behind the wait for the accumulator
            int32_t tgt = -1;
            float lse2 = 0.f, ratio = 0.f;
            const bool counts = (KIND == kDlogitsFew ? row & (kPaired - 1) : row) < count;
            if constexpr (KIND != kProducts) {
                if (KIND == kStats && p.direct) {  // one that does not count hits no column, or its value is not used
                    const int64_t y = row < count ? load_id(p.targets, p.is64, row) : -1;
                    tgt = y >= 0 && y < q.N ? (int32_t)y : -1;
                } else {
                    tgt = __ldcg(p.target + row);
                    if constexpr (KIND != kStats) tgt -= p.col0;
                }
                if constexpr (KIND == kDlogits || KIND == kDlogitsFew) {
                    lse2 = __ldcg(p.lse2 + row);
                    ratio = __ldcg(p.ratio + row);
                }
            }
            const uint32_t src = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * 128);
            // dz of the 32 columns of chunk c from their logits
            auto store_dz = [&](int c, const uint32_t (&z)[32]) {
                const int32_t col = c0 + c * 32, hit = tgt - col;
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float x[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float pr = exp2_approx(fmaf(__uint_as_float(z[2 * j + e]), kLog2e, -lse2));
                        x[e] = (2 * j + e == hit ? pr - 1.f : pr) * ratio;
                    }
                    w[j] = counts ? pack_bf16(x[0], x[1]) : 0u;
                    if (KIND == kDlogitsFew && row >= kPaired && counts)
                        w[j] = pack_bf16(x[0] - bf16_lo(w[j]), x[1] - bf16_hi(w[j]));
                }
                boxes.store(&q.map_c, lane, w, col, row0, col < q.N, false);
            };
            const bool runs = KIND == kStats || (KIND != kProducts && t.stages > run);
            if (runs) {
                // The logits are the sums of their runs' accumulators, added up here.
                uint32_t z[4][32];
                if constexpr (KIND != kStats) {  // added to from the first run on: reading that apart spilled
#pragma unroll
                    for (int j = 0; j < 128; ++j) z[j / 32][j % 32] = 0u;
                }
                for (int32_t i = 0; i < t.stages; i += run, ++tcount) {
                    const uint32_t ab = tcount & 1u;
                    if (!wait_bounded(&acc_full[ab], (tcount >> 1) & 1u, p.wait_ns, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (KIND == kStats && i == 0) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(src + ab * 256 + c * 32, z[c]);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c) {  // 8 columns at a time: 168 registers is the limit
                            uint32_t v[8];
                            tmem_ld_32x32b_x8(src + ab * 256 + c * 8, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                uint32_t& x = z[c / 4][(c & 3) * 8 + j];
                                x = __float_as_uint(__uint_as_float(x) + __uint_as_float(v[j]));
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_leader + ab * 8u);
                }
                if (!ok) break;
                if constexpr (KIND != kStats) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (half * 128 + c * 32 >= q.tile_n) break;  // past a narrow tile's columns
                        store_dz(c, z[c]);
                    }
                    continue;
                }
                asm volatile("" : "+r"(tgt));  // its load is not waited for earlier (8192 x 65536 x 256: 229 -> 213 us)
                if (!p.direct) tgt -= p.col0;
                float m = -INFINITY, sum = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int32_t col = c0 + c * 32;
                    // columns of this tile that are left: the vocabulary's end, or a narrow tile's
                    const int32_t left = min(q.N - t.n0, q.tile_n) - (half * 128 + c * 32);
                    if (left < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left) z[c][j] = 0xff800000u;
                    }
                    const int32_t hit = tgt - col;
                    if (hit >= 0 && hit < min(left, 32)) {
                        float x = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j == hit) x = __uint_as_float(z[c][j]);
                        p.target_logit[row] = x;
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) m = fmaxf(m, __uint_as_float(z[c][j]));
                }
                // all -inf: any finite reference leaves the terms 0
                const float ref = m == -INFINITY ? 0.f : m * kLog2e;
                float s4[4] = {};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        s4[j & 3] += exp2_approx(fmaf(__uint_as_float(z[c][j]), kLog2e, -ref));
                sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                // The terms are 2^(z log2 e - ref).  What rounding took from ref = m log2 e is put back, so that
                // the sum is that of exp(z - m): a confident token's loss is little more than its logarithm.
                if (m != -INFINITY) sum = fmaf(sum, -kLn2 * fmaf(m, kLog2e, -ref), sum);
                if (row < count)
                    p.stats[(int64_t)(t.n_tile * 2 + half) * p.rows + row] = make_float2(m, sum);
            } else {
                const uint32_t ab = tcount & 1u;
                if (!wait_bounded(&acc_full[ab], (tcount >> 1) & 1u, p.wait_ns, p.status)) break;
                ++tcount;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(src + ab * 256 + c * 32, v);
                    tmem_ld_wait();
                    if (c == 3) {  // the accumulator has been read out; the arrive only reports it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_leader + ab * 8u);
                    }
                    const int32_t col = c0 + c * 32;
                    if (half * 128 + c * 32 >= q.tile_n) continue;  // past a narrow tile's columns
                    if constexpr (KIND == kDlogits || KIND == kDlogitsFew) {
                        store_dz(c, v);
                    } else {
                        const int32_t y = t.slot * q.slot_rows + row0;
                        const bool in_m = q.m_counted || row0 < q.M;
                        if (q.scaled) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * gscale);
                        }
                        if (q.out_bf16) {
                            uint32_t w[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                w[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                            boxes.store(&q.map_c, lane, w, col, y, in_m && col < q.N, false);
                        } else {
                            boxes.store(&q.map_c, lane, v, col, y, in_m && col < q.N, q.add);
                            boxes.store(&q.map_c, lane, v + 16, col + 16, y, in_m && col + 16 < q.N, q.add);
                        }
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA frees TMEM or exits while the pair may still use it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- gather
constexpr int kGatherThreads = 512;
constexpr int kGatherWarps = kGatherThreads / 32;

struct GatherParams {
    const bf16* h;
    int64_t ldh;
    int32_t tokens, dim, vocab;
    int32_t paired;  // each row again kPaired rows further down
    int32_t vec;  // rows of h can be read in 16-byte vectors
    const void* targets;
    int32_t is64;
    int64_t ignore;
    int32_t reduction;
    // gradient only
    const float* lse;
    const float* dloss;
    // outputs
    Header* header;
    bf16* rows;        // [padded tokens][dim]
    int32_t* target;   // [padded tokens]
    int32_t* source;   // [padded tokens]: token of a gathered row
    int32_t* place;    // [tokens]: gathered row of a token, or -1
    float* lse2;
    float* ratio;
    float* loss;       // forward: zero for ignored tokens
    float* lse_out;
    uint32_t* status;
};

// The target of token t, or -1 when it does not count.
__device__ __forceinline__ int32_t counted_target(const GatherParams& p, int32_t t, bool report) {
    const int64_t y = load_id(p.targets, p.is64, t);
    if (y == p.ignore) return -1;
    if (y < 0 || y >= p.vocab) {
        if (report) atomicOr(p.status, kStatusBadIndex);
        return -1;
    }
    return (int32_t)y;
}

// Each CTA gathers a contiguous range of tokens.  Where its rows go follows from the number of
// counted tokens in front of them, which it counts by itself: the targets are short beside
// the rows, and no CTA waits for another.  8 to 10 us at 1531 tokens, latency.
template <bool GRAD>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
    __shared__ int32_t warp_n[2][kGatherWarps];
    __shared__ int32_t list_src[kGatherThreads];
    __shared__ int32_t n_list;
    grid_dependency_wait();
    allow_dependent_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t per = (p.tokens + (int32_t)gridDim.x - 1) / (int32_t)gridDim.x;
    const int32_t begin = (int32_t)min((int64_t)blockIdx.x * per, (int64_t)p.tokens);
    const int32_t end = (int32_t)min((int64_t)begin + per, (int64_t)p.tokens);

    int32_t before = 0, total = 0;
#pragma unroll 4
    for (int32_t t = tid; t < p.tokens; t += kGatherThreads) {
        const int32_t on = counted_target(p, t, blockIdx.x == 0) >= 0;
        total += on;
        before += t < begin ? on : 0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) warp_n[0][warp] = before, warp_n[1][warp] = total;
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int w = 0; w < kGatherWarps; ++w) before += warp_n[0][w], total += warp_n[1][w];

    if (blockIdx.x == 0 && tid == 0) {
        p.header->count = total;
        float g = 1.f;
        if (GRAD && p.reduction != MXFP4_REDUCE_NONE) {
            g = p.dloss[0];
            if (p.reduction == MXFP4_REDUCE_MEAN) g /= (float)max(total, 1);
        }
        p.header->gscale = g;
    }

    const int units = p.dim / 8;
    for (int32_t t0 = begin; t0 < end; t0 += kGatherThreads) {
        const int32_t t = t0 + tid;
        const int32_t y = t < end ? counted_target(p, t, false) : -1;
        const uint32_t on = __ballot_sync(0xffffffffu, y >= 0);
        __syncthreads();  // the counts and the list of the round before have been read
        if (lane == 0) warp_n[0][warp] = __popc(on);
        __syncthreads();
        int32_t lower = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kGatherWarps; ++w) {
            lower += w < warp ? warp_n[0][w] : 0;
            all += warp_n[0][w];
        }
        const int32_t at = lower + __popc(on & ((1u << lane) - 1));
        if (t < end) {
            p.place[t] = y >= 0 ? before + at : -1;
            if (y >= 0) {
                const int32_t r = before + at;
                list_src[at] = t;
                p.target[r] = y;
                p.source[r] = t;
                if constexpr (GRAD) {
                    const float l = p.lse[t] * kLog2e;
                    const float g = p.reduction == MXFP4_REDUCE_NONE ? p.dloss[t] : 1.f;
                    p.lse2[r] = l;
                    p.ratio[r] = g;
                    if (p.paired) {
                        p.target[r + kPaired] = y;
                        p.lse2[r + kPaired] = l;
                        p.ratio[r + kPaired] = g;
                    }
                }
            } else if constexpr (!GRAD) {
                p.lse_out[t] = 0.f;
                p.loss[t] = 0.f;
            }
        }
        if (tid == 0) n_list = all;
        __syncthreads();
        for (int32_t i = warp; i < n_list; i += kGatherWarps) {
            const bf16* src = p.h + (int64_t)list_src[i] * p.ldh;
            bf16* dst = p.rows + (int64_t)(before + i) * p.dim;
            for (int copy = 0; copy <= (GRAD ? p.paired : 0); ++copy, dst += (int64_t)kPaired * p.dim) {
                if (p.vec) {
#pragma unroll 8
                    for (int u = lane; u < units; u += 32)
                        reinterpret_cast<uint4*>(dst)[u] = reinterpret_cast<const uint4*>(src)[u];
                } else {
                    for (int c = lane; c < p.dim; c += 32) dst[c] = src[c];
                }
            }
        }
        before += all;
    }
    // Behind the counted rows: their dz is 0 up to the end of the last tile, whatever their logits are,
    // but rows that share dw's last stage with them are multiplied by that 0 and must be finite.
    const bool paired = GRAD && p.paired;
    const int32_t padded = paired ? kPaired : pad_rows(total);
    const int32_t stage_end = paired ? kPaired : (max(total, 1) + kK - 1) / kK * kK;
    for (int32_t r0 = total + (int32_t)blockIdx.x * kGatherWarps + warp; r0 < padded;
         r0 += (int32_t)gridDim.x * kGatherWarps)
        for (int32_t r = r0; r <= r0 + (paired ? kPaired : 0); r += kPaired) {
            if (GRAD && r0 < stage_end) {
                bf16* dst = p.rows + (int64_t)r * p.dim;
                for (int u = lane; u < units; u += 32) reinterpret_cast<uint4*>(dst)[u] = make_uint4(0, 0, 0, 0);
            }
            if (lane == 0) {
                p.target[r] = -1;
                if constexpr (GRAD) p.lse2[r] = 0.f, p.ratio[r] = 0.f;
            }
        }
}

// ---------------------------------------------------------------- combine
constexpr int kCombineThreads = 256;
constexpr int kCombineRows = 8;  // 64 bytes of each tile's statistics
constexpr int kCombineGroups = kCombineThreads / kCombineRows;

struct CombineParams {
    const Header* header;
    const float2* stats;
    int32_t parts, rows;
    const float* target_logit;
    const int32_t* source;
    float* lse;
    float* loss;
    // without a gather: the tokens' own targets decide what counts
    int32_t direct, tokens, vocab, is64;
    const void* targets;
    int64_t ignore;
    uint32_t* status;
};

// kCombineRows rows per CTA, a group of threads to each: the walk over the tiles is a chain of loads
// (8 rows x 286 statistics 8 us under ncu, most of it the launch and two trips to L2).
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p) {
    __shared__ float2 sh[kCombineThreads / 32][kCombineRows];
    grid_dependency_wait();
    allow_dependent_launch();
    int32_t count = p.tokens;
    if (!p.direct) count = counted_tokens(p.header);
    const int r = threadIdx.x % kCombineRows, g = threadIdx.x / kCombineRows;
    const int32_t row = blockIdx.x * kCombineRows + r;
    if ((int32_t)blockIdx.x * kCombineRows >= count) return;
    float m = -INFINITY, s = 0.f;
    auto join = [&](float2 o) {
        const float top = fmaxf(m, o.x);
        const float ref = top == -INFINITY ? 0.f : top;
        s = s * exp2_approx((m - ref) * kLog2e) + o.y * exp2_approx((o.x - ref) * kLog2e);
        m = top;
    };
    if (row < count) {
        constexpr int kFlight = 8;  // loads in flight
        for (int32_t i = g; i < p.parts; i += kFlight * kCombineGroups) {
            float2 o[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const int32_t at = i + k * kCombineGroups;
                o[k] = at < p.parts ? __ldcg(&p.stats[(int64_t)at * p.rows + row]) : make_float2(-INFINITY, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k) join(o[k]);
        }
    }
    // Groups are joined pairwise: lanes 8 and 16 apart, then the warps in order.
#pragma unroll
    for (int o = kCombineRows; o < 32; o <<= 1)
        join(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o)));
    if ((threadIdx.x & 31) < kCombineRows) sh[threadIdx.x >> 5][r] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x >= kCombineRows || row >= count) return;
    m = sh[0][r].x, s = sh[0][r].y;
#pragma unroll
    for (int k = 1; k < kCombineThreads / 32; ++k) join(sh[k][r]);
    const float ln_s = logf(s);
    float lse = m + ln_s, loss = 0.f;
    int32_t t = row;
    bool counts = true;
    if (p.direct) {
        const int64_t y = load_id(p.targets, p.is64, row);
        counts = y != p.ignore && y >= 0 && y < p.vocab;
        if (!counts && y != p.ignore) atomicOr(p.status, kStatusBadIndex);
    } else {
        t = p.source[row];
    }
    if (counts)
        loss = (m - p.target_logit[row]) + ln_s;  // exact difference where the target is the largest
    else
        lse = 0.f;
    p.lse[t] = lse;
    p.loss[t] = loss;
}

// Sum or mean of the tokens' losses, in one CTA: a fixed order.
constexpr int kReduceThreads = 1024;
__global__ void __launch_bounds__(kReduceThreads)
    reduce_kernel(const CombineParams p, int32_t mean, float* out) {
    __shared__ float warp_sum[kReduceThreads / 32];
    grid_dependency_wait();
    allow_dependent_launch();
    float s = 0.f;
#pragma unroll 4
    for (int32_t t = threadIdx.x; t < p.tokens; t += kReduceThreads) s += __ldcg(p.loss + t);
    int32_t count = 0;
    if (!p.direct) {
        count = counted_tokens(p.header);
    } else if (mean) {  // at most one tile of tokens, and the CTA has more threads
        bool on = false;
        if (threadIdx.x < p.tokens) {
            const int64_t y = load_id(p.targets, p.is64, threadIdx.x);
            on = y != p.ignore && y >= 0 && y < p.vocab;
        }
        count = __syncthreads_count(on);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = warp_sum[threadIdx.x];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) out[0] = mean ? s / (float)max(count, 1) : s;
    }
}

// ---------------------------------------------------------------- scatter
constexpr int kScatterThreads = 256;

// dh[t] = gscale * sum over the parts of row place[t]; one warp per token and 256 columns.
template <class DH>
__global__ void __launch_bounds__(kScatterThreads)
    scatter_kernel(const Header* header, const int32_t* place, const float* parts, int32_t splits, int64_t slot_elems,
                   int32_t tokens, int32_t dim, uint32_t segs, DH* dh, int64_t lddh, int32_t vec, int32_t paired) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t wid = (int64_t)blockIdx.x * (kScatterThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = wid / segs;
    const int32_t u = (int32_t)(wid - t * segs) * 32 + (threadIdx.x & 31);
    if (t >= tokens || u * 8 >= dim) return;
    const int32_t r = place[t];
    const float gscale = shared_factor(header);
    float v[8] = {};
    if (r >= 0) {
        const float* src = parts + (int64_t)r * dim + u * 8;
        for (int half = 0; half <= paired; ++half, src += (int64_t)kPaired * dim)
#pragma unroll 4
            for (int32_t k = 0; k < splits; ++k) {
                float x[8];
                unpack8(load8(src + k * slot_elems), x);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += x[j];
            }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= gscale;
    }
    DH* dst = dh + t * lddh + u * 8;
    if (vec) {
        store8(dst, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) store1(dst + j, v[j]);
    }
}

// ---------------------------------------------------------------- host
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The dz of one piece: at most this many bytes (or kMinPiece columns), so that a long batch
// needs no more scratch than a short one.  A piece's products are then long enough that the ends of
// their launches cost little: of 8192 tokens of a 128256 x 512 layer the gradients take 2258 us with pieces
// of 256 MB, 2107 with 512 and 1994 with 1024.  (Pieces of 48 MB, whose dz would stay in L2, were slower
// throughout: 65536 x 256, 759 us against 1301.)
constexpr size_t kPieceBytes = size_t(512) << 20;
constexpr int32_t kMinPiece = 2048;

int32_t piece_columns(int32_t padded, int64_t vocab) {
    const int64_t fit = std::max<int64_t>(kMinPiece, (int64_t)(kPieceBytes / (2 * (size_t)padded)) / kTile * kTile);
    const int64_t pieces = (vocab + fit - 1) / fit;
    const int64_t even = (vocab + pieces - 1) / pieces;
    return (int32_t)((even + kTile - 1) / kTile * kTile);
}

// Parts that dh's contraction over a piece's columns is cut into, so that its few long tiles fill the
// device beside dw's many short ones.  A schedule takes the parts' own rounds, or all tiles' stages
// shared out; a part costs two stages of hand-off and twelve for the passes over its fp32 output.  How
// many tokens count is known on the device alone, so the number is taken whose schedule is best
// where all of them do (twice) and half of them (once), each against one that is shared out evenly.
// Lowered to the parts that get work; every piece uses at most as many.
int32_t split_count(int32_t padded, int64_t dim, int32_t columns) {
    const int64_t n_tiles = (dim + kTile - 1) / kTile;
    const int64_t w_tiles = (columns + kTile - 1) / kTile * n_tiles;
    const int32_t stages = (columns + kK - 1) / kK;
    int32_t best = 1;
    double best_cost = 1e30;
    for (int32_t s = 1; s <= 16 && s <= stages; ++s) {
        const int64_t per = (stages + s - 1) / s;
        double cost = 0;
        for (int32_t share = 1; share <= 2; ++share) {
            const int32_t rows = pad_rows(padded / share);
            const int64_t tiles = rows / kTile * n_tiles, others = w_tiles * (std::max(rows / kK, 6) + 2);
            const int64_t rounds = (tiles * s + kClustersMost - 1) / kClustersMost * (per + 2);
            const int64_t shared = (tiles * s * (per + 14) + others) / kClustersMost;
            const int64_t even = (tiles * (stages + 14) + others) / kClustersMost + 1;
            cost += (double)std::max(rounds, shared) / (double)even / share;
        }
        if (cost < best_cost) best = s, best_cost = cost;
    }
    const int32_t per = (stages + best - 1) / best;
    return (stages + per - 1) / per;
}

struct Layout {
    int32_t padded;
    size_t header, target, source, place, lse2, ratio, target_logit, token_loss, rows, stats, dz, parts, bytes;
    int32_t tile_n;  // of the forward pass
    int32_t piece, splits;
};

Layout lay_out(int64_t tokens, int64_t vocab, int64_t dim, bool grad) {
    Layout l{};
    l.padded = pad_rows((int32_t)tokens);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    const size_t n = (size_t)l.padded;
    l.header = take(sizeof(Header));
    l.target = take(n * 4);
    l.source = take(n * 4);
    l.place = take(n * 4);
    l.rows = take(n * (size_t)dim * 2);
    if (!grad) {
        l.target_logit = take(n * 4);
        l.token_loss = take(n * 4);
        l.tile_n = vocab_tile(l.padded / kTile, vocab, dim);
        l.stats = take((size_t)((vocab + l.tile_n - 1) / l.tile_n) * 2 * n * sizeof(float2));
    } else {
        l.lse2 = take(n * 4);
        l.ratio = take(n * 4);
        l.piece = piece_columns(l.padded, vocab);
        l.splits = split_count(l.padded, dim, (int32_t)std::min<int64_t>(l.piece, vocab));
        l.dz = take(n * (size_t)l.piece * 2);
        l.parts = take((size_t)l.splits * n * (size_t)dim * 4);
    }
    l.bytes = at;
    return l;
}

// The kernels count rows, columns and tiles in 32 bits.
bool sizes_fit(int64_t tokens, int64_t vocab, int64_t dim) {
    return tokens >= 0 && vocab >= 0 && dim >= 0 && tokens <= (1 << 24) && vocab <= (1 << 28) && dim <= (1 << 16) &&
           ((tokens + kTile - 1) / kTile) * ((vocab + 127) / 128) <= (1 << 30);
}

template <int KIND>
cudaError_t launch_matrix(const CeParams& p, int64_t tiles, cudaStream_t s) {
    auto kern = ce_matrix_kernel<KIND>;
    static DeviceSlots slots;
    int clusters = 0;
    cudaError_t e = per_device_setting(slots, &clusters, [&](int dev, int* n) {
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (r != cudaSuccess) return r;
        int sms = 0;
        r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (r != cudaSuccess) return r;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t probe = {};
        probe.gridDim = dim3((unsigned)(sms & ~1));
        probe.blockDim = dim3(kThreads);
        probe.dynamicSmemBytes = kSmem;
        probe.attrs = attr;
        probe.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(n, kern, &probe);
    });
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorNotSupported;
    const int64_t grid = 2 * std::min<int64_t>(tiles, clusters);
    return launch_overlapped(kern, dim3((unsigned)grid), dim3(kThreads), kSmem, s, 2, true, p);
}

int64_t tiles_of(int64_t m, int64_t n, int64_t width) { return ((m + kTile - 1) / kTile) * ((n + width - 1) / width); }

// Eight tokens to a CTA, two CTAs an SM; for a gradient's few tokens more CTAs share the zero rows behind them.
cudaError_t gather_grid(int64_t tokens, int least, int* grid) {
    static DeviceSlots slots;
    int sms = 0;
    cudaError_t e = per_device_setting(
        slots, &sms, [&](int dev, int* n) { return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev); });
    *grid = (int)std::min<int64_t>(2 * sms, std::max<int64_t>(least, (tokens + 7) / 8));
    return e;
}

// Checks what the two calls share.  *empty: there is no token or no element.
mxfp4_status check_common(const char* what, const void* h, int64_t tokens, int64_t dim, int64_t ldh, const void* w,
                          int64_t vocab, int64_t ldw, const void* targets, int ids_dtype, int reduction) {
    if (tokens < 0 || vocab < 0 || dim < 0) return record_error(MXFP4_ERR_INVALID_ARG, "%s: negative size", what);
    if (ids_dtype != MXFP4_IDS_I32 && ids_dtype != MXFP4_IDS_I64)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad ids_dtype %d", what, ids_dtype);
    if (reduction < MXFP4_REDUCE_NONE || reduction > MXFP4_REDUCE_MEAN)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad reduction %d", what, reduction);
    if (vocab == 0 || dim == 0)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: vocab and dim must be positive", what);
    if (dim % 8) return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: dim (%lld) %% 8 != 0", what, (long long)dim);
    if (!sizes_fit(tokens, vocab, dim))
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: more than 2^24 tokens, 2^28 ids, 2^16 columns or 2^45 logits", what);
    if (!w) return record_error(MXFP4_ERR_INVALID_ARG, "%s: w is NULL", what);
    if (reinterpret_cast<uintptr_t>(w) % 16 || ldw % 8)
        return record_error(MXFP4_ERR_MISALIGNED, "%s: w must be 16-byte aligned with ldw %% 8 == 0", what);
    if (ldw < dim) return record_error(MXFP4_ERR_INVALID_ARG, "%s: ldw below dim", what);
    if (tokens == 0) return MXFP4_OK;
    if (!h || !targets) return record_error(MXFP4_ERR_INVALID_ARG, "%s: h or targets is NULL", what);
    if (ldh < dim) return record_error(MXFP4_ERR_INVALID_ARG, "%s: ldh below dim", what);
    if (reinterpret_cast<uintptr_t>(h) % 2 ||
        reinterpret_cast<uintptr_t>(targets) % (ids_dtype == MXFP4_IDS_I64 ? 8 : 4))
        return record_error(MXFP4_ERR_MISALIGNED, "%s: h or targets not aligned to its type", what);
    return MXFP4_OK;
}

mxfp4_status check_ws(const char* what, const void* ws, size_t have, size_t need) {
    if (!ws || have < need) return record_error(MXFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", what, need);
    if (reinterpret_cast<uintptr_t>(ws) % 256)
        return record_error(MXFP4_ERR_MISALIGNED, "%s: workspace not 256-byte aligned", what);
    return MXFP4_OK;
}

mxfp4_status launch_failed(const char* what, const char* step, cudaError_t e) {
    return record_error(MXFP4_ERR_CUDA, "%s: %s: %s", what, step, cudaGetErrorString(e));
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mxfp4_linear_ce_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
    if (tokens <= 0 || vocab <= 0 || dim <= 0 || !sizes_fit(tokens, vocab, dim)) return 0;
    return lay_out(tokens, vocab, dim, false).bytes;
}

extern "C" size_t mxfp4_linear_ce_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
    if (tokens <= 0 || vocab <= 0 || dim <= 0 || !sizes_fit(tokens, vocab, dim)) return 0;
    return lay_out(tokens, vocab, dim, true).bytes;
}

extern "C" mxfp4_status mxfp4_linear_ce(const void* h, int64_t tokens, int64_t dim, int64_t ldh, const void* w,
                                        int64_t vocab, int64_t ldw, const void* targets, int ids_dtype,
                                        int64_t ignore_index, int reduction, float* loss, float* lse, void* ws,
                                        size_t ws_bytes, mxfp4_stream_t stream) {
    const char* what = "linear_ce";
    mxfp4_status st = check_common(what, h, tokens, dim, ldh, w, vocab, ldw, targets, ids_dtype, reduction);
    if (st) return st;
    const bool reduced = reduction != MXFP4_REDUCE_NONE;
    if (tokens > 0 || reduced) {
        if (!loss || (tokens > 0 && !lse)) return record_error(MXFP4_ERR_INVALID_ARG, "%s: loss or lse is NULL", what);
        if ((reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(lse)) % 4)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: loss or lse misaligned", what);
    }
    if (tokens > 0 && (st = check_ws(what, ws, ws_bytes, mxfp4_linear_ce_workspace_bytes(tokens, vocab, dim)))) return st;
    if (tokens == 0 && !reduced) return record_error(MXFP4_OK, "%s", "");
    if ((st = ensure_device())) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0) {
        const cudaError_t e = cudaMemsetAsync(loss, 0, sizeof(float), s);
        return e != cudaSuccess ? launch_failed(what, "clear", e) : record_error(MXFP4_OK, "%s", "");
    }
    const Layout l = lay_out(tokens, vocab, dim, false);
    uint8_t* base = static_cast<uint8_t*>(ws);
    float* token_loss = reduced ? reinterpret_cast<float*>(base + l.token_loss) : loss;
    const int is64 = ids_dtype == MXFP4_IDS_I64;
    // One tile of tokens that TMA can read: gathering would cost a launch (5 of 31 us for 7 tokens of
    // a 32000 x 1024 layer) and save no tile.
    const bool direct = tokens <= kTile && vector_rows(h, ldh, dim, 2);
    Header* header = reinterpret_cast<Header*>(base + l.header);

    CeParams p{};
    Product& q = p.prod[0];
    bf16* rows = reinterpret_cast<bf16*>(base + l.rows);
    if (!(direct ? encode_bf16_map(&q.map_a, h, tokens, dim, ldh, kK, 128)
                 : encode_bf16_map(&q.map_a, rows, l.padded, dim, dim, kK, 128)) ||
        !encode_bf16_map(&q.map_b, w, vocab, dim, ldw, kK, (uint32_t)l.tile_n / 2))
        return record_error(MXFP4_ERR_CUDA, "%s: tensor map encoding failed", what);
    q.m_counted = 1;
    q.M = l.padded;
    q.N = (int32_t)vocab;
    q.tile_n = l.tile_n;
    q.num_n = (q.N + q.tile_n - 1) / q.tile_n;
    q.tx = stage_bytes(l.tile_n);
    q.K = (int32_t)dim;
    q.splits = 1;
    p.count = 1;
    p.header = header;
    p.target = reinterpret_cast<int32_t*>(base + l.target);
    p.direct = direct;
    p.tokens = (int32_t)tokens;
    p.is64 = is64;
    p.targets = targets;
    p.rows = l.padded;
    p.stats = reinterpret_cast<float2*>(base + l.stats);
    p.target_logit = reinterpret_cast<float*>(base + l.target_logit);
    p.status = device_status_ptr();
    p.wait_ns = wait_limit_ns();

    cudaError_t e;
    if (!direct) {
        GatherParams g{};
        g.h = static_cast<const bf16*>(h);
        g.ldh = ldh;
        g.tokens = (int32_t)tokens;
        g.dim = (int32_t)dim;
        g.vocab = (int32_t)vocab;
        g.vec = vector_rows(h, ldh, dim, 2);
        g.targets = targets;
        g.is64 = is64;
        g.ignore = ignore_index;
        g.reduction = reduction;
        g.header = header;
        g.rows = rows;
        g.target = reinterpret_cast<int32_t*>(base + l.target);
        g.source = reinterpret_cast<int32_t*>(base + l.source);
        g.place = reinterpret_cast<int32_t*>(base + l.place);
        g.loss = token_loss;
        g.lse_out = lse;
        g.status = p.status;
        int grid = 1;
        e = gather_grid(tokens, 1, &grid);
        if (e == cudaSuccess)
            e = launch_overlapped(gather_kernel<false>, dim3(grid), dim3(kGatherThreads), 0, s, 1, true, g);
        if (e != cudaSuccess) return launch_failed(what, "gather", e);
    }
    e = launch_matrix<kStats>(p, tiles_of(l.padded, vocab, l.tile_n), s);
    if (e != cudaSuccess) return launch_failed(what, "statistics", e);
    CombineParams c{};
    c.header = header;
    c.stats = p.stats;
    c.parts = (int32_t)((vocab + l.tile_n - 1) / l.tile_n) * 2;
    c.rows = l.padded;
    c.target_logit = p.target_logit;
    c.source = reinterpret_cast<int32_t*>(base + l.source);
    c.lse = lse;
    c.loss = token_loss;
    c.direct = direct;
    c.tokens = (int32_t)tokens;
    c.vocab = (int32_t)vocab;
    c.is64 = is64;
    c.targets = targets;
    c.ignore = ignore_index;
    c.status = p.status;
    e = launch_overlapped(combine_kernel, dim3((unsigned)((tokens + kCombineRows - 1) / kCombineRows)),
                          dim3(kCombineThreads), 0, s, 1, true, c);
    if (e != cudaSuccess) return launch_failed(what, "combine", e);
    if (reduced) {
        e = launch_overlapped(reduce_kernel, dim3(1), dim3(kReduceThreads), 0, s, 1, true, c,
                              (int32_t)(reduction == MXFP4_REDUCE_MEAN), loss);
        if (e != cudaSuccess) return launch_failed(what, "reduce", e);
    }
    return record_error(MXFP4_OK, "%s", "");
}

extern "C" mxfp4_status mxfp4_linear_ce_grad(const void* h, int64_t tokens, int64_t dim, int64_t ldh, const void* w,
                                             int64_t vocab, int64_t ldw, const void* targets, int ids_dtype,
                                             int64_t ignore_index, int reduction, const float* lse, const float* dloss,
                                             void* dh, int dh_dtype, int64_t lddh, void* dw, int dw_dtype,
                                             int64_t lddw, int accumulate, void* ws, size_t ws_bytes,
                                             mxfp4_stream_t stream) {
    const char* what = "linear_ce_grad";
    mxfp4_status st = check_common(what, h, tokens, dim, ldh, w, vocab, ldw, targets, ids_dtype, reduction);
    if (st) return st;
    for (int t : {dh ? dh_dtype : 0, dw ? dw_dtype : 0})
        if (t != MXFP4_OUT_F32 && t != MXFP4_OUT_BF16)
            return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad output dtype %d", what, t);
    if (accumulate != 0 && accumulate != 1)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: accumulate must be 0 or 1", what);
    if (dw && accumulate && dw_dtype != MXFP4_OUT_F32)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: accumulate needs fp32 output", what);
    const int64_t hsz = dh_dtype == MXFP4_OUT_BF16 ? 2 : 4, wsz = dw_dtype == MXFP4_OUT_BF16 ? 2 : 4;
    if (dw) {
        if (lddw < dim) return record_error(MXFP4_ERR_INVALID_ARG, "%s: lddw below dim", what);
        if (reinterpret_cast<uintptr_t>(dw) % 16 || lddw * wsz % 16)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: dw must be 16-byte aligned with rows of 16 bytes", what);
    }
    if (tokens > 0) {
        if (!lse || !dloss) return record_error(MXFP4_ERR_INVALID_ARG, "%s: lse or dloss is NULL", what);
        if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(dloss)) % 4)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: lse or dloss misaligned", what);
        if (dh && lddh < dim) return record_error(MXFP4_ERR_INVALID_ARG, "%s: lddh below dim", what);
        if (dh && reinterpret_cast<uintptr_t>(dh) % hsz)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: dh not aligned to its type", what);
        if ((dh || dw) &&
            (st = check_ws(what, ws, ws_bytes, mxfp4_linear_ce_grad_workspace_bytes(tokens, vocab, dim))))
            return st;
    }
    if ((!dh && !dw) || (tokens == 0 && (!dw || accumulate))) return record_error(MXFP4_OK, "%s", "");
    if ((st = ensure_device())) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (tokens == 0) {
        e = cudaMemset2DAsync(dw, (size_t)(lddw * wsz), 0, (size_t)(dim * wsz), (size_t)vocab, s);
        return e != cudaSuccess ? launch_failed(what, "clear", e) : record_error(MXFP4_OK, "%s", "");
    }
    const Layout l = lay_out(tokens, vocab, dim, true);
    uint8_t* base = static_cast<uint8_t*>(ws);

    GatherParams g{};
    g.h = static_cast<const bf16*>(h);
    g.ldh = ldh;
    g.tokens = (int32_t)tokens;
    g.dim = (int32_t)dim;
    g.vocab = (int32_t)vocab;
    g.paired = tokens <= kPaired;
    g.vec = vector_rows(h, ldh, dim, 2);
    g.targets = targets;
    g.is64 = ids_dtype == MXFP4_IDS_I64;
    g.ignore = ignore_index;
    g.reduction = reduction;
    g.lse = lse;
    g.dloss = dloss;
    g.header = reinterpret_cast<Header*>(base + l.header);
    g.rows = reinterpret_cast<bf16*>(base + l.rows);
    g.target = reinterpret_cast<int32_t*>(base + l.target);
    g.source = reinterpret_cast<int32_t*>(base + l.source);
    g.place = reinterpret_cast<int32_t*>(base + l.place);
    g.lse2 = reinterpret_cast<float*>(base + l.lse2);
    g.ratio = reinterpret_cast<float*>(base + l.ratio);
    g.status = device_status_ptr();
    int grid = 1;
    e = gather_grid(tokens, 32, &grid);
    if (e == cudaSuccess)
        e = launch_overlapped(gather_kernel<true>, dim3(grid), dim3(kGatherThreads), 0, s, 1, true, g);
    if (e != cudaSuccess) return launch_failed(what, "gather", e);

    bf16* dz = reinterpret_cast<bf16*>(base + l.dz);
    float* parts = reinterpret_cast<float*>(base + l.parts);
    for (int64_t v0 = 0; v0 < vocab; v0 += l.piece) {
        const int32_t cols = (int32_t)std::min<int64_t>(l.piece, vocab - v0);
        const uint8_t* w_piece = static_cast<const uint8_t*>(w) + v0 * ldw * 2;
        CeParams p{};
        p.header = g.header;
        p.target = g.target;
        p.col0 = (int32_t)v0;
        p.rows = l.padded;
        p.paired = g.paired;
        p.lse2 = g.lse2;
        p.ratio = g.ratio;
        p.status = g.status;
        p.wait_ns = wait_limit_ns();
        {
            Product& q = p.prod[0];
            q.m_counted = 1;
            q.M = l.padded;
            q.N = cols;
            q.tile_n = vocab_tile(l.padded / kTile, cols, dim);
            q.num_n = (q.N + q.tile_n - 1) / q.tile_n;
            q.tx = stage_bytes(q.tile_n);
            q.K = (int32_t)dim;
            q.splits = 1;
            q.out_bf16 = 1;
            if (!encode_bf16_map(&q.map_a, g.rows, l.padded, dim, dim, kK, 128) ||
                !encode_bf16_map(&q.map_b, w_piece, cols, dim, ldw, kK, (uint32_t)q.tile_n / 2) ||
                !encode_out_map(&q.map_c, dz, l.padded, cols, l.piece, true))
                return record_error(MXFP4_ERR_CUDA, "%s: tensor map encoding failed", what);
            p.count = 1;
            e = p.paired ? launch_matrix<kDlogitsFew>(p, tiles_of(l.padded, cols, q.tile_n), s)
                         : launch_matrix<kDlogits>(p, tiles_of(l.padded, cols, q.tile_n), s);
            if (e != cudaSuccess) return launch_failed(what, "dlogits", e);
        }
        int n = 0;
        int64_t tiles = 0;
        if (dh) {  // the longer contraction first: the schedule ends on the shorter tiles
            Product& q = p.prod[n++];
            q = Product{};
            q.m_counted = 1;
            q.b_mn = 1;
            q.M = l.padded;
            q.N = (int32_t)dim;
            q.tile_n = even_tile(dim);
            q.num_n = (q.N + q.tile_n - 1) / q.tile_n;
            q.tx = stage_bytes(kTile);
            q.K = cols;
            const int32_t stages = (cols + kK - 1) / kK;
            q.k_per_split = (stages + l.splits - 1) / l.splits;
            q.splits = (stages + q.k_per_split - 1) / q.k_per_split;
            q.slot_rows = l.padded;
            q.add = v0 > 0;
            if (!encode_bf16_map(&q.map_a, dz, l.padded, cols, l.piece, kK, 128) ||
                !encode_bf16_map(&q.map_b, w_piece, cols, dim, ldw, 64, kK) ||
                !encode_out_map(&q.map_c, parts, (int64_t)l.splits * l.padded, dim, dim, false))
                return record_error(MXFP4_ERR_CUDA, "%s: tensor map encoding failed", what);
            tiles += tiles_of(l.padded, dim, q.tile_n) * q.splits;
        }
        if (dw) {
            Product& q = p.prod[n++];
            q = Product{};
            q.a_mn = q.b_mn = 1;
            q.k_counted = 1;
            q.M = cols;
            q.N = (int32_t)dim;
            q.tile_n = even_tile(dim);
            q.num_n = (q.N + q.tile_n - 1) / q.tile_n;
            q.tx = stage_bytes(kTile);
            q.K = l.padded;
            q.splits = 1;
            q.scaled = 1;
            q.out_bf16 = dw_dtype == MXFP4_OUT_BF16;
            q.add = accumulate;
            if (!encode_bf16_map(&q.map_a, dz, l.padded, cols, l.piece, 64, kK) ||
                !encode_bf16_map(&q.map_b, g.rows, l.padded, dim, dim, 64, kK) ||
                !encode_out_map(&q.map_c, static_cast<uint8_t*>(dw) + v0 * lddw * wsz, cols, dim, lddw, q.out_bf16))
                return record_error(MXFP4_ERR_CUDA, "%s: tensor map encoding failed", what);
            tiles += tiles_of(cols, dim, q.tile_n);
        }
        p.count = n;
        e = launch_matrix<kProducts>(p, tiles, s);
        if (e != cudaSuccess) return launch_failed(what, "products", e);
    }
    if (dh) {
        const uint32_t segs = (uint32_t)((dim / 8 + 31) / 32);
        const int64_t blocks = (tokens * segs + kScatterThreads / 32 - 1) / (kScatterThreads / 32);
        const int64_t slot = (int64_t)l.padded * dim;
        if (dh_dtype == MXFP4_OUT_BF16)
            e = launch_overlapped(scatter_kernel<bf16>, dim3((unsigned)blocks), dim3(kScatterThreads), 0, s, 1, true,
                                  (const Header*)g.header, (const int32_t*)g.place, (const float*)parts, l.splits, slot,
                                  (int32_t)tokens, (int32_t)dim, segs, static_cast<bf16*>(dh), lddh,
                                  (int32_t)vector_rows(dh, lddh, dim, 2), g.paired);
        else
            e = launch_overlapped(scatter_kernel<float>, dim3((unsigned)blocks), dim3(kScatterThreads), 0, s, 1, true,
                                  (const Header*)g.header, (const int32_t*)g.place, (const float*)parts, l.splits, slot,
                                  (int32_t)tokens, (int32_t)dim, segs, static_cast<float*>(dh), lddh,
                                  (int32_t)vector_rows(dh, lddh, dim, 4), g.paired);
        if (e != cudaSuccess) return launch_failed(what, "scatter", e);
    }
    return record_error(MXFP4_OK, "%s", "");
}
