// Definitions shared by the paged cache's translation units: the workspace,
// row addresses, the e4m3 conversions and the small matrix instructions.
#pragma once

#include "wf_internal.cuh"

namespace wf {

// ----------------------------------------------------------------- workspace
// control block | arrival counters (zero at rest) | pages that a reserve call
// copies | shared items and partial results of the attention's splits
constexpr int PA_TILE_M = 16;       // query heads of a single-token item at most
constexpr int PA_MAX_CTAS = 640;    // most CTAs of a single-token launch
constexpr int PA_MAX_ROUND_CTAS = 160;   // and of a launch over drafted rows
constexpr int PA_ROUND_M = 256;     // pairs of an item there

struct PagedLayout {
    size_t cnt, n_copies, copies, join, stat, part, total;
};

// The counters have a fixed place, sized for the most sequences: calls of
// different shapes share a workspace and none writes where another counts.
// Partial results: two partials of a tile for each CTA.
inline PagedLayout paged_layout(int D, int max_rows) {
    constexpr size_t SEQS = WF_PAGED_MAX_SEQS;
    static_assert(SEQS >= PA_MAX_CTAS, "a counter for each CTA");
    const size_t token = (size_t)PA_MAX_CTAS * 2 * PA_TILE_M, rounds = (size_t)PA_MAX_ROUND_CTAS * 2 * PA_ROUND_M;
    const size_t rows = max_rows > 1 && rounds > token ? rounds : token;
    PagedLayout L;
    size_t o = sizeof(Control);
    L.cnt = o;
    o = align_up(o + 4 * SEQS, 256);
    L.n_copies = o;   // pages listed by the current reserve launch
    o += 256;
    L.copies = o;
    o = align_up(o + 8 * SEQS, 256);
    L.join = o;
    o = align_up(o + 16 * (size_t)PA_MAX_ROUND_CTAS, 256);
    L.stat = o;
    o = align_up(o + 8 * rows, 256);
    L.part = o;
    o = align_up(o + 4 * rows * (size_t)D, 256);
    L.total = o;
    return L;
}

// ----------------------------------------------------------------- conversions
__device__ __forceinline__ uint16_t pg_f32_to_bf16(float f) {   // nearest even; NaN stays NaN
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7F800000u) == 0x7F800000u && (u & 0x007FFFFFu)) return (uint16_t)((u >> 16) | 0x40u);
    u += 0x7FFFu + ((u >> 16) & 1u);
    return (uint16_t)(u >> 16);
}
__device__ __forceinline__ float pg_bf16_to_f32(uint32_t b) { return __uint_as_float(b << 16); }
// (lo, hi) -> two bf16 / fp16 in one word, round to nearest even
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// the same, rounded toward zero
__device__ __forceinline__ uint32_t cvt_bf16x2_down(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// (lo, hi) -> two e4m3 bytes, saturating, round to nearest even
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// two e4m3 bytes (the low half of w) -> two fp16, exact
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

// fp16 queries: a row whose largest element is `big` is divided by 2^e, which
// puts it in [1, 2) (a row of zeros or subnormals lower).  Within +-126 both 2^e
// and 2^-e are normal numbers; bf16's largest exponent, 127, leaves [2, 4).
__device__ __forceinline__ int pg_scale_exponent(float big) {
    return min(max((int)(__float_as_uint(big) >> 23) - 127, -126), 126);
}
// The factor that turns such a row's products into base-2 exponents.  Never 0,
// which would make NaN of a masked score (-inf); products below it are nothing.
__device__ __forceinline__ float pg_factor(float s, int e) {
    const float f = s * __uint_as_float((uint32_t)(127 + e) << 23);
    return f < 1e-37f ? 1e-37f : f;
}

// largest base-2 exponent that stands for itself in fp32: rounded by 1/32 at most
constexpr float PG_FAR = 1048576.f;

// ----------------------------------------------------------------- matrix instructions
__device__ __forceinline__ void pg_mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void pg_mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void pg_ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void pg_ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// 16 bytes global -> shared; `bytes` = 0 writes zeros and reads nothing
__device__ __forceinline__ void pg_cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void pg_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// a / b of numbers that are seldom past 32 bits, b > 0
__device__ __forceinline__ int64_t pg_quotient(int64_t a, int64_t b) {
    if (((uint64_t)a | (uint64_t)b) >> 32 == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Last sequence whose first row is at or before row p: the largest b with
// off[b] <= p, or -1 (warp-collective, the same answer in every lane).  Each
// step loads 32 samples, so 1,024 sequences take two dependent loads.
__device__ __forceinline__ int warp_seq_of(const int32_t* off, int B, int p, int lane) {
    int lo = 0, n = B;   // candidates [lo, lo + n)
    if (off[0] > p) return -1;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool le = i < n && off[lo + i] <= p;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int s = m ? 31 - __clz(m) : 0;
        lo += s * step;
        n = min(step, n - s * step);
    }
    return lo;
}

}  // namespace wf
