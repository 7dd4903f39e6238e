// step_ops.cuh -- what the step operators' translation units (embedding, linear cross
// entropy, gradient clipping) share beside internal.h and ptx.cuh: a status bit, host helpers
// of mxfp4_api.cu and further inline PTX.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace mx {

// Status bit: a token id or target outside the vocabulary (and not the ignored / padding one).
constexpr uint32_t kStatusBadIndex = 4u;

// ------------------------------------------------------------------ host (mxfp4_api.cu)
mxfp4_status ensure_device();  // current device checked (GB300), status word looked up, context bound
uint64_t wait_limit_ns();      // this thread's bounded-wait limit
// 2D tensor map over a row-major bf16 matrix [rows, cols] (leading dimension ld elements):
// box = box_cols x box_rows, 128-byte swizzle, zero fill outside.
bool encode_bf16_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, uint32_t box_cols,
                     uint32_t box_rows);

// ------------------------------------------------------------------ device
// Waits until the shared-memory sources of all but the N most recently committed bulk groups
// have been read.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// bf16 operands (kind::f16), fp32 accumulation, issued for a CTA pair.
__device__ __forceinline__ void tc_mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor for kind::f16 with bf16 A/B and fp32 accumulation.  a_mn / b_mn: that
// operand's M (N) index runs along its shared-memory rows instead of K.
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
    return (1u << 4)                // D format: fp32
           | (1u << 7)              // A format: bf16
           | (1u << 10)             // B format: bf16
           | (a_mn << 15) | (b_mn << 16)
           | ((N >> 3) << 17)       // N / 8
           | ((M >> 4) << 24);      // M / 16
}

// TMEM -> registers: 32 lanes (this warp's sub-partition) x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// 2^x (ex2.approx: about 2 ulp, 2^-inf = 0, subnormal results flushed).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace mx
