// What the target head's log-probabilities and the draft head's distillation
// share: one sweep of a head's weights over the rows, whose logits are folded
// as they leave the accumulator, and the merge of the sweep's partial states.
#pragma once

#include "wf_pipe.cuh"

namespace wf {

static_assert(WF_MAX_LISTED <= 64, "a warp's lanes take two listed ids each");
constexpr int PICK_NONE = 0x7fffffff;    // a list's place without an id: matches nothing

// Rows swept by one launch: what they read stays in L2 while the weights
// stream past, and the states of a launch have a bounded size.
constexpr long SWEEP_ACT_BYTES = 48L << 20;
constexpr int SWEEP_MAX_ROWS = 16384;
inline int sweep_chunk(int rows, int d) {
    long c = SWEEP_ACT_BYTES / (2L * d) / (2 * BM) * (2 * BM);
    if (c > SWEEP_MAX_ROWS) c = SWEEP_MAX_ROWS;
    return rows < c ? rows : (int)c;   // d <= 16,384: at least 1,536 rows
}

// The state that one CTA (or pair) leaves for a row: (M, S, T, 0) as in
// state_merge, then the k best as (logit, id) words.
__host__ __device__ constexpr size_t state_bytes(int kt) { return 16 + 8 * (size_t)kt; }
// Lists of two widths.  10 for up to 10: 16 for all of them take 536 us where this
// takes 521 (1,248 rows of 2,560 over 151,936 ids, 10 best), 163 for 134 (2,000 of 256
// over 40,000, 4 best).  A third width of 4 would take 104 there and 516 for 527 with
// one best over the large head; not built.
inline int state_width(int k) { return k == 0 ? 0 : k <= 10 ? 10 : 16; }
constexpr int REACHED = 16;              // words for the maxima of a row that the pairs of a sweep share
constexpr int STATE_SLOTS = 160;         // CTAs of a sweep of one activation tile
// (pairs of a sweep of several: REC_PAIRS)
inline size_t states_bytes(int rows, int d, int k) {
    // no fewer for more rows, so that a workspace for the most rows serves fewer
    const size_t many = (size_t)sweep_chunk(rows, d) * REC_PAIRS, few = (size_t)(rows < BM ? rows : BM) * STATE_SLOTS;
    return (many > few ? many : few) * state_bytes(state_width(k));
}

struct SweepCall {
    const uint16_t *act, *W;
    int rows, d, V;          // rows: of this launch, at most sweep_chunk()
    float inv_t;
    const int32_t* pick;     // [rows][K] ids in any order, or null
    int K;
    float* picked;           // [rows][K] their logits, where the id lies in [0, V)
    uint8_t* states;
    int k;                   // best logits kept
    uint32_t* reached;       // scratch [rows][REACHED], 16-byte aligned (k > 0)
    bool entropy;
    float* z;                // [rows][ldz] logits times inv_t, or null
    int64_t ldz;
    bool after_lists;        // the kernel before on the stream is this call's that made the lists
    Control* ctrl;
};
// Enqueues the sweep; *slots: states left for each row (row-major, in use all of them).
wf_status launch_sweep(const SweepCall& c, int* slots, cudaStream_t s);

// A teacher's alternatives.
struct Teacher {
    const int32_t* tid;      // [N][K]
    const float* tlogit;     // [N][K]
    const int32_t* t2d;      // [V] or null: tid are draft ids
    int N, K, V, Vd;
    float inv_t;
    Control* ctrl;
};
// ... as lists for a sweep: ids [N][K] draft ids (PICK_NONE: not kept), p their
// probabilities, stat [N] sum p log p (NaN: an id out of range).
wf_status launch_teacher(const Teacher& t, int32_t* ids, float* p, float* stat, cudaStream_t s);

struct MergeCall {
    const uint8_t* states;   // [rows][slots]
    int rows, slots, k, K;
    float inv_t;
    float* lse;              // [rows] or null
    float* H;                // [rows] or null
    int32_t* top_ids;        // [rows][k] or null
    float* top_logp;         // [rows][k] or null
    const float* picked;     // [rows][K]
    const int32_t* ids;      // [rows][K] as swept
    float* logp;             // [rows][K] or null
    float* loss;             // [rows] or null; then either the lists as launch_teacher made them
    const float* p;          // [rows][K]
    const float* stat;       // [rows]
    const float* z;          // or [rows][ldz], the logits that the sweep kept, and the teacher
    int64_t ldz;
    Teacher t;
    int V;
    int row0;                // first row's number in the call, for errors
    Control* ctrl;
};
wf_status launch_states_merge(const MergeCall& c, cudaStream_t s);

// (M, S, T) of two states of one row: M the largest logit, S = sum 2^z, T = sum
// z 2^z, z = c (v - M).  The difference comes first: the largest logit has z = 0
// and S >= 1 whatever c M's size is (a rounded c M in place of it is off by more
// than 2^z can take once c M passes 2^31, a small temperature's).  A state with
// S = 0 is empty; NaN stays NaN.
__device__ __forceinline__ void state_merge(float c, float& M, float& S, float& T, float m2, float s2, float t2) {
    if (s2 == 0.f) return;
    if (S == 0.f) {
        M = m2;
        S = s2;
        T = t2;
        return;
    }
    const float mx = fmaxf(M, m2);
    const float d1 = (M - mx) * c, d2 = (m2 - mx) * c;
    const float a1 = ex2_approx(d1), a2 = ex2_approx(d2);
    // a state far below the other: its weight is 0, and so is its part of T
    T = (a1 == 0.f && S == S ? 0.f : (T + d1 * S) * a1) + (a2 == 0.f && s2 == s2 ? 0.f : (t2 + d2 * s2) * a2);
    S = S * a1 + s2 * a2;
    M = mx;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
// NaN wins
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = v != v || o <= v ? v : o;
    }
    return v;
}

// One row's alternatives by one warp: lane l has places l and l + 32.
struct TeacherRow {
    int id[2];      // draft id, PICK_NONE for a place that is not kept
    float p[2];     // softmax of the kept logits / T; entries of one id stay apart
    float plogp;    // sum p log p; NaN if an id is out of range
    bool some;      // whether the row has a kept alternative
};
__device__ __forceinline__ TeacherRow teacher_row(const Teacher& t, int row, int lane) {
    const size_t base = (size_t)row * t.K;
    TeacherRow r;
    float l[2];
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        r.id[h] = PICK_NONE;
        l[h] = -INFINITY;
        if (j < t.K) {
            int v = t.tid[base + j];
            const float logit = t.tlogit[base + j];
            bool none = v == -1;
            if (!none && t.t2d) {
                if (v < 0 || v >= t.V) {
                    bad = true;
                    none = true;
                } else {
                    v = t.t2d[v];
                    none = v < 0;   // no draft id for this target id
                }
            }
            if (!none && (v < 0 || v >= t.Vd)) {
                bad = true;
                none = true;
            }
            if (!none && logit != -INFINITY) {
                l[h] = logit;
                r.id[h] = v;
            }
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad) {   // the row takes no part
        r.id[0] = r.id[1] = PICK_NONE;
        l[0] = l[1] = -INFINITY;
        if (lane == 0) record_error(t.ctrl, WF_ERR_BAD_DATA, (uint32_t)row);
    }
    const float top = warp_max(l[0] != l[0] || l[1] <= l[0] ? l[0] : l[1]);
    r.some = top != -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) r.p[h] = r.some && r.id[h] != PICK_NONE ? expf((l[h] - top) * t.inv_t) : 0.f;
    const float total = warp_sum(r.p[0] + r.p[1]);
    float plogp = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (r.some && r.id[h] != PICK_NONE) {
            // log p from the logits: a p that rounds to 0 has a finite logarithm, times 0
            const float logp = (l[h] - top) * t.inv_t - logf(total);
            r.p[h] /= total;
            plogp += r.p[h] == 0.f ? 0.f : r.p[h] * logp;
        }
    }
    r.plogp = bad ? __int_as_float(0x7fc00000) : warp_sum(plogp);
    return r;
}

}  // namespace wf
