// The pipelined tcgen05 product that the heads' scoring and training kernels
// share: a shared-memory ring filled by TMA, one elected thread issuing the
// MMAs into two TMEM accumulators, and epilogue warps that read them.
//
//   warp 0     fills the ring: each stage holds an A tile and a B tile of one K
//              block (64 values of K), copied by one elected thread
//   warp 1     allocates TMEM and issues the MMAs of a stage (one elected
//              thread); the stage is free again when they have completed
//   warps 2-   read a finished accumulator (thread = one row of the tile, or of
//              one half of its columns) while the next tile's MMAs run into the
//              other one
// PAIR: the two CTAs of a cluster compute one 256-row tile with paired MMAs;
// each loads its own half of A's rows and of B's, the first CTA issues, and
// both CTAs' barriers are committed to.
// Every mbarrier wait is bounded: one that runs out records WF_ERR_TIMEOUT, raises
// the CTA's abort flag, waits (again bounded) for its own copies and MMAs in
// flight, and the CTA frees TMEM and exits.
// The other waits have no limit of their own; what each waits for does not wait
// for it:
//   TMEM (pipe_begin)   CTAs that hold some on this SM, of whatever kernel or
//                       stream, give it back when their own work is done.  The
//                       CTAs of a pair allocate one by one, so two pairs that had
//                       one SM of the same two each would wait for one another:
//                       a pair's CTA takes more than half of an SM's shared
//                       memory (asserted beside each kernel, as the LM head's
//                       pairs do), so no SM ever holds CTAs of two pairs.
//   cluster barriers    both CTAs of a pair are started together, and every thread
//                       reaches both barriers, also behind a wait that gave up
//   pdl_wait            the kernel before, which waits for nothing (stream order,
//                       below)
//   bulk-store groups   copies out of this CTA's own shared memory
#pragma once

#include "wf_internal.cuh"

namespace wf {

// Threads with `w` epilogue warps (4 or 8: a warp reads the 32 accumulator rows that its number mod 4 gives).
constexpr int pipe_threads(int w) { return 64 + 32 * w; }
constexpr int PIPE_MAX_STAGES = 12;
constexpr int PIPE_TMEM_COLS = 2 * BN;     // two fp32 accumulators of up to BN columns
constexpr int PIPE_BARRIER_BYTES = 512;    // barriers, TMEM address and abort flag behind the ring
constexpr int PIPE_SMEM_MAX = 227 * 1024;  // a CTA's shared memory
constexpr int PIPE_STATIC_MAX = 512;       // of it, for a kernel's static shared memory
// Whether no SM (228 KB, 1 KB of it reserved for each CTA) holds two CTAs of this much dynamic shared memory.
constexpr bool pipe_alone(int smem) { return 2 * (smem + 1024) > 228 * 1024; }
// What a kernel records beside WF_ERR_TIMEOUT: which wait gave up.
constexpr uint32_t PIPE_WHERE_COPY = 0x400, PIPE_WHERE_ACC = 0x500, PIPE_WHERE_STAGE = 0x510, PIPE_WHERE_TILE = 0x600;

struct Pipe {
    uint8_t* base;                 // the ring, 1,024-byte aligned
    int stages, stage_bytes, a_bytes;
    uint64_t *full, *empty, *tfull, *tempty, *drain;
    uint32_t* tmem_slot;
    volatile int* abort_flag;
    Control* ctrl;
    uint64_t timeout_ns;
    __device__ __forceinline__ uint8_t* a(int s) const { return base + (size_t)s * stage_bytes; }
    __device__ __forceinline__ uint8_t* b(int s) const { return base + (size_t)s * stage_bytes + a_bytes; }
    __device__ __forceinline__ void fail(uint32_t where) const {
        *abort_flag = 1;
        record_error(ctrl, WF_ERR_TIMEOUT, where);
    }
};

// Ring, `extra` bytes (a multiple of 1,024) behind it and the barriers, in dynamic shared memory from its start
// rounded up to 1,024 bytes.
__device__ __forceinline__ Pipe pipe_at(uint8_t* smem_raw, int stages, int stage_bytes, int a_bytes, int extra,
                                        Control* ctrl, uint64_t timeout_ns) {
    Pipe g;
    g.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    g.stages = stages;
    g.stage_bytes = stage_bytes;
    g.a_bytes = a_bytes;
    g.full = reinterpret_cast<uint64_t*>(g.base + (size_t)stages * stage_bytes + extra);
    g.empty = g.full + PIPE_MAX_STAGES;
    g.tfull = g.empty + PIPE_MAX_STAGES;
    g.tempty = g.tfull + 2;
    g.drain = g.tempty + 2;
    g.tmem_slot = reinterpret_cast<uint32_t*>(g.drain + 1);
    g.abort_flag = reinterpret_cast<volatile int*>(g.tmem_slot + 1);
    g.ctrl = ctrl;
    g.timeout_ns = timeout_ns;
    return g;
}
__device__ __forceinline__ uint8_t* pipe_extra(const Pipe& g) { return g.base + (size_t)g.stages * g.stage_bytes; }
constexpr int pipe_smem(int stages, int stage_bytes, int extra) {
    return stages * stage_bytes + PIPE_BARRIER_BYTES + extra + 1024;
}

// The thread's warp, the same in all of its lanes also to the compiler.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// Barriers and TMEM; returns the TMEM base address.  All threads.
template <bool PAIR, int EPI_WARPS>
__device__ __forceinline__ uint32_t pipe_begin(const Pipe& g) {
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(&g.full[s], 1);
            mbar_init(&g.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&g.tfull[a], 1);
            mbar_init(&g.tempty[a], (PAIR ? 2 : 1) * EPI_WARPS);   // PAIR: both CTAs' epilogue warps release
        }
        mbar_init(g.drain, 1);
        *g.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(g.tmem_slot, PIPE_TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(g.tmem_slot, PIPE_TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();   // both CTAs' barriers and TMEM exist before either uses the other's
    tc_fence_after();
    return __shfl_sync(0xffffffffu, *g.tmem_slot, 0);
}

template <bool PAIR>
__device__ __forceinline__ void pipe_end(const Pipe& g, uint32_t tmem_base) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();   // the first CTA's MMAs and the second's remote arrivals are done
    tc_fence_after();
    if ((threadIdx.x >> 5) == 1) {
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem_base, PIPE_TMEM_COLS);
        else
            tmem_dealloc(tmem_base, PIPE_TMEM_COLS);
    }
}

// One thread of the warp, the same one every time (all lanes).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// The copying warp (all lanes).  next(i) sets up the CTA's i-th tile and returns
// its K blocks (0: no further tile); tx() is what a stage of it receives in bytes
// (PAIR: both CTAs together); load(kc, s, bar, a, b) issues the copies of operand
// A (if a) and B (if b) into stage s, counted on the barrier at shared address
// `bar` (PAIR: the first CTA's), by one elected thread, the warp walking the loop
// together as in pipe_mma.
// EARLY: B is a weight matrix, whose first stages are asked for while the kernel
// before (of the same call, which has itself waited for what came before it) is
// still running; everything else waits for it.
template <bool PAIR, bool EARLY, typename Next, typename Tx, typename Load>
__device__ __forceinline__ void pipe_copy(const Pipe& g, bool first, Next next, Tx tx, Load load) {
    const uint32_t full0 = PAIR ? cluster_addr(&g.full[0], 0) : smem_u32(&g.full[0]);
    auto bar = [&](int s) { return full0 + (uint32_t)(s * sizeof(uint64_t)); };
    auto fill = [&](int kc, int s, uint32_t bytes, bool fresh, bool a, bool b) {
        if (elect_one()) {
            if (fresh && (!PAIR || first)) mbar_arrive_expect_tx(&g.full[s], bytes);
            load(kc, s, bar(s), a, b);
        }
        __syncwarp();
    };
    int num_k = next(0);
    uint32_t bytes = tx();
    int early = 0;
    if constexpr (EARLY) {
        early = num_k < g.stages ? num_k : g.stages;
        for (int s = 0; s < early; ++s) {
            fill(s, s, bytes, true, false, true);
        }
    }
    pdl_wait();
    uint32_t it = 0;   // stages issued so far
    int s = 0;         // = it % stages
    uint32_t ph = 0;   // = (it / stages) & 1
    bool ok = true;
    for (int i = 0; ok && num_k > 0;) {
        for (int kc = 0; kc < num_k; ++kc, ++it) {
            if (it > 0 && ++s == g.stages) {
                s = 0;
                ph ^= 1;
            }
            // the lanes give up a wait together
            if (!__all_sync(0xffffffffu, mbar_wait(&g.empty[s], ph ^ 1, g.timeout_ns, g.abort_flag))) {
                g.fail(PIPE_WHERE_COPY + s);
                ok = false;
                break;
            }
            const bool fresh = !EARLY || it >= (uint32_t)early;
            fill(kc, s, bytes, fresh, true, fresh);
        }
        num_k = next(++i);
        bytes = tx();
    }
    // the last stages' releases have arrived too before the CTA's shared memory is another's
    for (uint32_t j = (it > (uint32_t)g.stages ? it - g.stages : 0); ok && j < it; ++j)
        ok = __all_sync(0xffffffffu, mbar_wait(&g.empty[j % g.stages], (j / g.stages) & 1, g.timeout_ns, g.abort_flag));
    if (!ok || __any_sync(0xffffffffu, *g.abort_flag)) {
        // let every copy this warp issued land before the CTA exits
        if (!PAIR || first) {
            for (uint32_t j = (it > (uint32_t)g.stages ? it - g.stages : 0); j < it; ++j)
                mbar_wait(&g.full[j % g.stages], (j / g.stages) & 1, g.timeout_ns, nullptr);
        } else {
            // the second CTA's copies are counted on the first CTA's barriers,
            // which it cannot wait on: give them a fixed 200 us (a copy from L2
            // or HBM takes a few)
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000ull) {
            }
        }
    }
}

// The issuing warp (all lanes; PAIR: of the first CTA).  next(i) as above;
// issue(s, d_tmem, kc) issues stage s's MMAs into the accumulator at d_tmem (kc =
// 0 overwrites it), by one elected thread.  The warp walks the loop together and
// only the issue itself is one thread's: the compiler then knows the operands to be
// the warp's, where a lane in a branch of its own took 70 cycles for each MMA (645
// a stage whose products take 512: 1,248 rows of 2,560 over 151,936 ids 558 us a
// call, 500 so).
template <bool PAIR, typename Next, typename Issue>
__device__ __forceinline__ void pipe_mma(const Pipe& g, uint32_t tmem_base, Next next, Issue issue) {
    const uint32_t empty_peer = PAIR ? cluster_addr(&g.empty[0], 1) : 0;
    const uint32_t tfull_peer = PAIR ? cluster_addr(&g.tfull[0], 1) : 0;
    uint32_t it = 0;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true, issued = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, g.timeout_ns, g.abort_flag)) != 0;
    };
    for (uint32_t i = 0; ok; ++i) {
        const int num_k = next((int)i);
        if (num_k == 0) break;
        const uint32_t acc = i & 1, acc_ph = (i >> 1) & 1;
        // PAIR: released by both CTAs' epilogues (the second's arrivals are remote)
        if (!wait(&g.tempty[acc], acc_ph ^ 1)) {
            g.fail(PIPE_WHERE_ACC);
            ok = false;
            break;
        }
        tc_fence_after();
        for (int kc = 0; kc < num_k; ++kc, ++it) {
            if (it > 0 && ++s == g.stages) {
                s = 0;
                ph ^= 1;
            }
            if (!wait(&g.full[s], ph)) {
                g.fail(PIPE_WHERE_STAGE + s);
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                issue(s, tmem_base + acc * BN, kc);
                if constexpr (PAIR) {
                    umma_commit_pair(smem_u32(&g.empty[s]));
                    umma_commit_pair(empty_peer + (uint32_t)(s * sizeof(uint64_t)));
                } else {
                    umma_commit(&g.empty[s]);
                }
            }
            __syncwarp();
            issued = true;
        }
        if (ok && elect_one()) {
            if constexpr (PAIR) {
                umma_commit_pair(smem_u32(&g.tfull[acc]));
                umma_commit_pair(tfull_peer + acc * (uint32_t)sizeof(uint64_t));
            } else {
                umma_commit(&g.tfull[acc]);
            }
        }
    }
    if (issued && (!ok || PAIR)) {
        // every MMA issued above (PAIR: into both CTAs' TMEM) has completed before TMEM is freed
        uint64_t* drain = g.drain;
        if (elect_one()) {
            if constexpr (PAIR)
                umma_commit_pair(smem_u32(drain));
            else
                umma_commit(drain);
        }
        __syncwarp();
        mbar_wait(drain, 0, g.timeout_ns, nullptr);
    }
}

// Epilogue warps (all lanes): wait for the i-th accumulator, and hand it back.
// The lanes leave the wait, or give it up, together: what follows (accumulator
// reads, votes) is for whole warps.
__device__ __forceinline__ bool pipe_acc_wait(const Pipe& g, uint32_t i) {
    __syncwarp();
    const bool there = mbar_wait(&g.tfull[i & 1], (i >> 1) & 1, g.timeout_ns, g.abort_flag);
    if (!__all_sync(0xffffffffu, there)) {
        g.fail(PIPE_WHERE_TILE);
        return false;
    }
    tc_fence_after();
    __syncwarp();
    return true;
}
// tempty_first: in a pair's second CTA the shared::cluster address of the first CTA's accumulator barriers, else 0.
// One arrival a warp, without a fence at cluster scope: nothing in memory is handed over, and the accumulator's reads
// are ordered by tcgen05's own fences.  (A release at cluster scope waits for the warp's shared-memory writes on their
// way out: 1,850 cycles a tile.)
__device__ __forceinline__ void pipe_acc_release(const Pipe& g, uint32_t i, uint32_t tempty_first) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        if (tempty_first)
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                             tempty_first + (i & 1) * (uint32_t)sizeof(uint64_t))
                         : "memory");
        else
            mbar_arrive(&g.tempty[i & 1]);
    }
}

// One box into shared memory, its bytes counted on the barrier at `bar`.
template <bool PAIR>
__device__ __forceinline__ void pipe_load(uint8_t* dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                          uint64_t policy) {
    if constexpr (PAIR) {
        tma_load_2d_pair(dst, map, bar, x, y, policy);
    } else {
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
            : "memory");
    }
}

// One box out of shared memory (clipped at the tensor's ends), by one thread:
// the box has to have been made visible with fence_async_store first.
__device__ __forceinline__ void fence_async_store() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the newest `N` stores of this thread have read their shared memory / all stores are done.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Byte of 16-byte unit u of row r in a 128-byte-row tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int r, int u) { return (uint32_t)(r * 128 + ((u ^ (r & 7)) << 4)); }

// Tensor map of [rows, cols] with row stride `stride` (elements), read or
// written in boxes of box_cols (128 bytes) x box_rows, 128-byte swizzle.
bool make_tile_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t stride, bool fp32,
                   uint32_t box_cols, uint32_t box_rows);
// Stream order of these kernels.  A sweep or a product takes every SM nearly whole
// (all tensor memory, up to 226 KB of shared memory, CTA pairs that need both SMs of
// a pair free at once), so what follows one, and what begins a call, is launched in
// plain stream order.  Only the kernel straight before it in the same call (the
// lists, the pass that makes G) lets it start early.  That one was itself launched
// in plain order, so it is all that is unfinished on the stream; it waits for
// nothing; and it lets go in its first instruction, which takes effect when every
// one of its blocks has started, so that blocks which wait beside them keep none of
// it from running.
// (Where every kernel let the next one start early, long queues of steps stopped
// about once in 10,000 passes, with no bounded wait giving up.  Why is not
// established; in this order more than three million passes ran clean, in the same
// time.)
template <typename... KArgs, typename... Args>
inline wf_status launch_plain(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              unsigned cluster, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) == cudaSuccess ? WF_OK : WF_ERR_CUDA;
}

// Dynamic shared memory that a kernel may ask for, and SMs set up for as much shared memory as there is by every kernel
// of these calls, so that none is set up anew between them (where one was, a call took 3 to 15 us longer).
template <typename K>
inline bool set_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                cudaSharedmemCarveoutMaxShared) == cudaSuccess;
}
// Clusters of two CTAs of `kernel` that can be resident at once, at most REC_PAIRS.
int resident_pairs(const void* kernel, int threads, int smem);
constexpr int REC_PAIRS = 80;

}  // namespace wf
