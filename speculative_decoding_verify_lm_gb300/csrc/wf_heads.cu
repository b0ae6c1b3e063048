// The small kernels around a sweep of a head's weights: a teacher's alternatives
// as probabilities over draft ids, for the sweep to look for, and the merge of a
// row's states into its log-sum-exp, entropy, best alternatives,
// log-probabilities and loss.  Both are bound by latency, one row's chain of
// loads and votes: a merge takes 6 to 7.5 us at 17 to 1,024 rows (a full head's
// sweep of few rows 118).
#include "wf_heads.cuh"

namespace wf {

namespace {

constexpr int LIST_WARPS = 4;

// One warp a row.
__global__ void __launch_bounds__(LIST_WARPS * 32) teacher_kernel(const Teacher t, int32_t* ids, float* p,
                                                                  float* stat) {
    pdl_trigger();   // the sweep may start and ask for its first weights
    const int row = blockIdx.x * LIST_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= t.N) return;
    const TeacherRow r = teacher_row(t, row, lane);
    const size_t base = (size_t)row * t.K;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < t.K) {
            ids[base + lane + 32 * h] = r.id[h];
            p[base + lane + 32 * h] = r.p[h];
        }
    if (lane == 0) stat[row] = r.plogp;
}

// One CTA a row, one thread a state; a fixed order of merging makes the result
// the same in every run.  The states come out of L2 (17 rows: 152 of 16 to 144
// bytes a row).
constexpr int MERGE_WARPS = STATE_SLOTS / 32;   // as many of them as the row has states
static_assert(MERGE_WARPS * 32 >= STATE_SLOTS && MERGE_WARPS * 32 >= REC_PAIRS, "a thread for every state");

template <int KT>
__global__ void __launch_bounds__(MERGE_WARPS * 32) states_merge_kernel(const MergeCall c) {
    __shared__ float wm[MERGE_WARPS], wsum[MERGE_WARPS], wt[MERGE_WARPS];
    __shared__ uint64_t wbest[MERGE_WARPS * 16];
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const float cc = LOG2E * c.inv_t;
    float M = -INFINITY, S = 0.f, T = 0.f;
    uint64_t loc[KT > 0 ? KT : 1];   // the state's list, best first
#pragma unroll
    for (int j = 0; j < KT; ++j) loc[j] = 0;
    if ((int)threadIdx.x < c.slots) {
        const float4* at =
            reinterpret_cast<const float4*>(c.states + ((size_t)row * c.slots + threadIdx.x) * state_bytes(KT));
        const float4 h = at[0];
        float4 e[KT > 0 ? KT / 2 : 1];
#pragma unroll
        for (int j = 0; j < KT / 2; ++j) e[j] = at[1 + j];
        M = h.x;
        S = h.y;
        T = h.z;
#pragma unroll
        for (int j = 0; j < KT; ++j) {
            const float4 f = e[j / 2];
            const int id = __float_as_int(j & 1 ? f.w : f.y);
            // + 0: zeros of both signs are one value, and rank by id
            loc[j] = id < 0 ? 0ull : pack_key((j & 1 ? f.z : f.x) + 0.f, (uint32_t)id);
        }
    }
    // the teacher's chain of loads (ids, their draft ids, those logits) while the states are on their way
    TeacherRow r{};
    float zt[2] = {0.f, 0.f};
    if (c.z && warp == 0) {
        r = teacher_row(c.t, c.row0 + row, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (r.p[h] != 0.f) zt[h] = c.z[(size_t)row * c.ldz + r.id[h]];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, M, off), s2 = __shfl_xor_sync(0xffffffffu, S, off),
                    t2 = __shfl_xor_sync(0xffffffffu, T, off);
        // both lanes of a pair merge the lower lane's state first
        if (lane & off) {
            float m = m2, s = s2, t = t2;
            state_merge(cc, m, s, t, M, S, T);
            M = m;
            S = s;
            T = t;
        } else {
            state_merge(cc, M, S, T, m2, s2, t2);
        }
    }
    if (lane == 0) {
        wm[warp] = M;
        wsum[warp] = S;
        wt[warp] = T;
    }
    if constexpr (KT > 0) {
        // the warp's k best, one after the other: keys are unique, so one lane owns each
        for (int j = 0; j < c.k; ++j) {
            const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(loc[0] >> 32));
            const uint32_t lo =
                __reduce_max_sync(0xffffffffu, (uint32_t)(loc[0] >> 32) == hi ? (uint32_t)loc[0] : 0u);
            const uint64_t best = ((uint64_t)hi << 32) | lo;
            if (lane == 0) wbest[warp * c.k + j] = best;
            if (loc[0] == best) {
#pragma unroll
                for (int s = 0; s < KT - 1; ++s) loc[s] = loc[s + 1];
                loc[KT - 1] = 0;
            }
        }
    }
    __syncthreads();
    M = wm[0];
    S = wsum[0];
    T = wt[0];
    for (int w = 1; w < warps; ++w) state_merge(cc, M, S, T, wm[w], wsum[w], wt[w]);
    // The largest logit over the temperature is rounded as a kept one is, so that it cancels against it: in the loss
    // below, and where log S is lost in lse also in the gradients, which have z and lse alone.
    const float logs = logf(S), zmax = __fmul_rn(M, c.inv_t);
    auto logq = [&](float v) { return fmaf(v - M, c.inv_t, -logs); };
    if (threadIdx.x == 0) {
        if (c.lse) c.lse[row] = __fadd_rn(zmax, logs);
        if (c.H) c.H[row] = logs - T * LN2 / S;
    }
    if constexpr (KT > 0) {
        // each of the warps' winners finds its place among all of them
        const int n = warps * c.k;
        if ((int)threadIdx.x < n) {   // k <= 16 a warp: a thread for each
            const uint64_t key = wbest[threadIdx.x];
            int place = 0;
            for (int j = 0; j < n; ++j) place += wbest[j] > key || (wbest[j] == key && j < (int)threadIdx.x);
            if (place < c.k) {
                const size_t o = (size_t)row * c.k + place;
                if (c.top_ids) c.top_ids[o] = key ? (int32_t)key_id(key) : -1;
                if (c.top_logp)
                    c.top_logp[o] = key ? logq(key_val(key)) : __int_as_float(0x7fc00000);
            }
        }
    }
    if (c.logp) {
        for (int j = threadIdx.x; j < c.K; j += blockDim.x) {
            const size_t at = (size_t)row * c.K + j;
            const int id = c.ids[at];
            if (id >= 0 && id < c.V) {
                c.logp[at] = logq(c.picked[at]);
            } else {
                c.logp[at] = id == -1 ? 0.f : __int_as_float(0x7fc00000);
                if (id != -1) record_error(c.ctrl, WF_ERR_BAD_DATA, (uint32_t)(c.row0 + row));
            }
        }
    }
    if (c.loss && warp == 0) {
        // sum p (log p - log q)
        float part = 0.f, stat;
        if (c.z) {
            stat = r.plogp;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (r.p[h] != 0.f) part = fmaf(r.p[h], (zt[h] - zmax) - logs, part);
        } else {
            stat = c.stat[row];
            for (int j = lane; j < c.K; j += 32) {
                const size_t at = (size_t)row * c.K + j;
                const float p = c.p[at];
                if (p != 0.f) part = fmaf(p, logq(c.picked[at]), part);
            }
        }
        part = warp_sum(part);
        if (lane == 0) c.loss[row] = stat - part;
    }
}

}  // namespace

static wf_status configure() {
    static std::mutex mu;
    static bool attr_set[64] = {false};
    return configure_once(mu, attr_set, [] {
        return set_smem(teacher_kernel, 0) && set_smem(states_merge_kernel<0>, 0) &&
               set_smem(states_merge_kernel<10>, 0) && set_smem(states_merge_kernel<16>, 0);
    });
}

wf_status launch_teacher(const Teacher& t, int32_t* ids, float* p, float* stat, cudaStream_t s) {
    const wf_status st = configure();
    if (st != WF_OK) return st;
    return launch_plain(teacher_kernel, dim3(cdiv(t.N, LIST_WARPS)), dim3(LIST_WARPS * 32), 0, s, 1u, t, ids, p, stat);
}

wf_status launch_states_merge(const MergeCall& c, cudaStream_t s) {
    const wf_status st = configure();
    if (st != WF_OK) return st;
    const dim3 block(cdiv(c.slots, 32) * 32);
    switch (state_width(c.k)) {
        case 0: return launch_plain(states_merge_kernel<0>, dim3(c.rows), block, 0, s, 1u, c);
        case 10: return launch_plain(states_merge_kernel<10>, dim3(c.rows), block, 0, s, 1u, c);
        default: return launch_plain(states_merge_kernel<16>, dim3(c.rows), block, 0, s, 1u, c);
    }
}

}  // namespace wf
