// k_quant_evict.cu -- eviction from the 4-bit KV cache by accumulated weight.
//
// Of a pair's keys the first `sink` and the last `recent` stay; of the others
// the heaviest, ties to the lower slots.  A radix select over the ordered bits
// of acc (three digits) gives the threshold weight; the kept slots are listed
// and their rows moved.
//
// A pair whose slots fit a CTA's shared memory is selected by each of its CTAs
// for itself, and each moves a share of the rows: reading acc again costs less
// than cluster barriers (64 pairs of 1600 keys: 19 us of 30 were those).  A
// longer one is a cluster's: each CTA has a run of slots, their histograms are
// joined through distributed shared memory, and their counts of kept keys and
// ties give each its places.  A run of up to kQeTile slots is read from HBM
// once; a longer one is read again for each digit.  Instructions bound the
// select, so every step takes 4 slots a lane.  The order of the rows is kept,
// so the result does not depend on the split.
#include <cooperative_groups.h>

#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace cg = cooperative_groups;

namespace pk {

constexpr int kQeThreads = 512;
constexpr int kQeWarps = kQeThreads / 32;
constexpr int kQeBins = 2048;            // digits of 11, 10 and 11 bits
constexpr int kQeTile = 16384;           // slots in shared memory: two CTAs to an SM
constexpr int kQeMaxCluster = 8;

struct QeSmem {
    uint32_t key[kQeTile];               // weights as they come, then their keys
    uint16_t list[kQeTile];              // kept slots of the tile, from its first on
    uint32_t hist[kQeBins];              // this CTA's counts
    uint32_t sums[kQeBins];              // all CTAs' counts; afterwards the marks of 4 slots each: bits 0..3 those that
                                         // stay, 4..7 those that tie
    uint32_t ws[kQeWarps + 1];
    uint32_t digit, left;
    uint32_t count[2];                   // kept and tied slots of this CTA
    unsigned long long bar;              // bulk copies of a tile
};
static_assert(kQeTile == 32 * kQeThreads, "a thread has one group of a tile");
static_assert(kQeTile / 4 <= kQeBins * 4, "the marks fit the sums");

// ordered bits of a weight; NaN sorts below everything
__device__ __forceinline__ uint32_t weight_key(float x)
{
    return x != x ? 0u : ord_f32(x + 0.0f);
}

// Rows i0 + list[j] of src to slots o0 + j of dst, j < count, by the CTA's
// warps: 32 rows at a time, 16 bytes a lane.
__device__ __forceinline__ void move_rows(const QuantEvictArgs &a, int p, int64_t i0, const uint16_t *list, int count, int64_t o0)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint8_t *src = a.src.blocks + (int64_t)p * (a.src.n_cap / kQKeys) * kQBlock;
    uint8_t *dst = a.dst.blocks + (int64_t)p * (a.dst.n_cap / kQKeys) * kQBlock;
    const float *acc = a.src.acc + (int64_t)p * a.src.n_cap;
    for (int j0 = 32 * warp; j0 < count; j0 += kQeThreads) {
        const int m = min(32, count - j0);
        uint4 kc[4], vc[4];
        uint2 ks = make_uint2(0, 0), vs = ks;
        float w = 0.0f;
        int slot = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {        // rows 8i + lane / 4, quarter lane % 4
            const int j = 8 * i + (lane >> 2);
            if (j < m) {
                const int x = (int)i0 + list[j0 + j];
                const uint8_t *b = src + (int64_t)(x / kQKeys) * kQBlock + x % kQKeys * kQRow;
                kc[i] = __ldcs(reinterpret_cast<const uint4 *>(b) + (lane & 3));
                // chunk places of V differ by the turn of the slot: taken in the order of slots with no turn
                vc[i] = __ldcs(reinterpret_cast<const uint4 *>(b + kQOffV) + ((lane & 3) ^ (v_turn(x) >> 1)));
            }
        }
        if (lane < m) {
            slot = (int)i0 + list[j0 + lane];
            const uint8_t *b = src + (int64_t)(slot / kQKeys) * kQBlock;
            ks = *reinterpret_cast<const uint2 *>(b + kQOffKs + 8 * (slot % kQKeys));
            vs = *reinterpret_cast<const uint2 *>(b + kQOffVs + 8 * (slot % kQKeys));
            if (a.dst.acc) w = acc[slot];
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int j = 8 * i + (lane >> 2);
            if (j < m) {
                const int64_t o = o0 + j0 + j;
                const int y = (int)(o % kQKeys);
                uint8_t *b = dst + o / kQKeys * kQBlock + y * kQRow;
                reinterpret_cast<uint4 *>(b)[lane & 3] = kc[i];
                reinterpret_cast<uint4 *>(b + kQOffV)[(lane & 3) ^ (v_turn(y) >> 1)] = vc[i];
            }
        }
        if (lane < m) {
            const int64_t o = o0 + j0 + lane;
            uint8_t *b = dst + o / kQKeys * kQBlock;
            *reinterpret_cast<uint2 *>(b + kQOffKs + 8 * (o % kQKeys)) = ks;
            *reinterpret_cast<uint2 *>(b + kQOffVs + 8 * (o % kQKeys)) = vs;
            if (a.dst.acc) a.dst.acc[p * a.dst.n_cap + o] = w;
            if (a.keep) a.keep[p * a.budget + o] = slot;
        }
    }
}

template <bool ALONE>
__global__ void __launch_bounds__(kQeThreads, 2) k_quant_evict(QuantEvictArgs a)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    QeSmem &sm = *reinterpret_cast<QeSmem *>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int p = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ALONE ? 0 : (int)cluster.block_rank(), ranks = ALONE ? 1 : (int)cluster.num_blocks();
    auto sync = [&]() { if (ALONE) __syncthreads(); else cluster.sync(); };
    if (tid == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"((uint32_t)__cvta_generic_to_shared(&sm.bar)) : "memory");
    }
    uint32_t phase = 0;
    bool late = false;
    pdl_wait();
    const int n = quant_len(a.src, p);
    if (blockIdx.x == 0 && tid == 0 && quant_len_bad(a.src, p)) quant_devchk(a.src.status, p);
    const float *acc = a.src.acc + (int64_t)p * a.src.n_cap;
    const bool vec = (uintptr_t)acc % 16 == 0;       // n_cap is a multiple of 32: the same for every pair
    const bool all = n <= a.budget;
    const int lo = all ? n : (int)a.sink, hi = all ? n : n - (int)a.recent;   // contested slots
    const uint32_t need = all ? 0u : (uint32_t)(a.budget - a.sink - a.recent);
    // this CTA's slots [c0, c1)
    const int run = (int)((((int64_t)n + ranks - 1) / ranks + 3) / 4 * 4);
    const int c0 = (int)min((int64_t)n, (int64_t)rank * run), c1 = min(n, c0 + run);
    int held = -1;                                   // first slot of the tile in shared memory
    // The weights of a tile to shared memory, by bulk copies where they are aligned: all its bytes are on their way at
    // once, and no register waits for them.
    auto bring = [&](int c, int m) {
        const int bulk = vec ? m / 4 * 4 : 0;
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncthreads();                             // the tile before is no longer read
        if (bulk) {
            const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&sm.bar);
            if (tid == 0) {
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(4 * bulk) : "memory");
                for (int i = 0; i < bulk; i += 4096)
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                     (uint32_t)__cvta_generic_to_shared(sm.key + i)),
                                 "l"(acc + c + i), "r"(4 * min(4096, bulk - i)), "r"(bar)
                                 : "memory");
            }
            bool done = false;
            for (int i = 0; i < (1 << 22) && !done; i++) {       // bounded
                uint32_t ok;
                asm volatile(
                    "{\n.reg .pred p;\n"
                    "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                    "selp.u32 %0, 1, 0, p;\n}\n"
                    : "=r"(ok)
                    : "r"(bar), "r"(phase)
                    : "memory");
                done = ok;
            }
            if (!done) late = true;
            phase ^= 1u;
        }
        for (int i = bulk + tid; i < m; i += kQeThreads) sm.key[i] = __float_as_uint(acc[c + i]);
        if (bulk < m) __syncthreads();
    };
    // 4 keys at slot i of the tile in shared memory; `fresh`: still weights
    auto keys = [&](uint32_t k[4], int i, bool fresh) {
        const uint4 v = *reinterpret_cast<const uint4 *>(sm.key + i);
        k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        if (fresh) {
#pragma unroll
            for (int e = 0; e < 4; e++) k[e] = weight_key(__uint_as_float(k[e]));
            *reinterpret_cast<uint4 *>(sm.key + i) = make_uint4(k[0], k[1], k[2], k[3]);
        }
    };

    // threshold key: the need-th largest of the contested; left: how many of those equal to it stay
    uint32_t prefix = 0, left = need;
    if (need) {
#pragma unroll 1
        for (int d = 0; d < 3; d++) {
            const int shift = d == 0 ? 21 : d == 1 ? 11 : 0, bins = d == 1 ? kQeBins / 2 : kQeBins;
            const uint32_t above = d == 0 ? 0u : d == 1 ? 0xffe00000u : 0xfffff800u;
            for (int i = tid; i < bins; i += kQeThreads) sm.hist[i] = 0;
            __syncthreads();
            for (int c = c0; c < c1; c += kQeTile) {
                const int m = min(kQeTile, c1 - c), first = lo - c, end = min(m, hi - c);
                const bool fresh = held != c;
                if (fresh) bring(c, m);
#pragma unroll 4
                for (int i = 4 * tid; i < m; i += 4 * kQeThreads) {
                    uint32_t k[4];
                    keys(k, i, fresh);
                    auto count = [&](int e) { atomicAdd(&sm.hist[(k[e] >> shift) & (bins - 1)], 1u); };
                    if (i >= first && i + 4 <= end) {
                        if (d == 0) {
#pragma unroll
                            for (int e = 0; e < 4; e++) count(e);
                            continue;
                        }
                        bool any = false;            // few agree with the digits before
#pragma unroll
                        for (int e = 0; e < 4; e++) any |= (k[e] & above) == prefix;
                        if (!any) continue;
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (i + e >= first && i + e < end && (k[e] & above) == prefix) count(e);
                }
                held = c;
            }
            sync();
            if (!ALONE) {                // each CTA joins the counts of its share of the bins and gives all the sums
                const int share = bins / ranks;
                for (int i = tid; i < share; i += kQeThreads) {
                    uint32_t x[kQeMaxCluster], v = 0;
#pragma unroll
                    for (int w = 0; w < kQeMaxCluster; w++) x[w] = w < ranks ? cluster.map_shared_rank(sm.hist, w)[rank * share + i] : 0u;
#pragma unroll
                    for (int w = 0; w < kQeMaxCluster; w++) v += x[w];
#pragma unroll
                    for (int w = 0; w < kQeMaxCluster; w++)
                        if (w < ranks) cluster.map_shared_rank(sm.sums, w)[rank * share + i] = v;
                }
                cluster.sync();
            }
            const uint32_t *sums = ALONE ? sm.hist : sm.sums;
            // thread t has bins [per t, per (t + 1))
            const int per = bins / kQeThreads;
            uint32_t mine[4] = {0, 0, 0, 0}, total = 0;
            for (int e = 0; e < per; e++) mine[e] = sums[per * tid + e];
            total = mine[0] + mine[1] + mine[2] + mine[3];
            uint32_t sum;
            uint32_t over = block_excl_scan<kQeThreads>(total, sm.ws, &sum);
            over = sum - over - total;               // keys in the bins above the thread's
#pragma unroll
            for (int e = 3; e >= 0; e--) {
                if (over < left && over + mine[e] >= left) {
                    sm.digit = per * tid + e;
                    sm.left = left - over;
                }
                over += mine[e];
            }
            __syncthreads();
            prefix |= sm.digit << shift;
            left = sm.left;
            __syncthreads();
        }
    }
    // marks of a tile
    auto mark = [&](int c) {
        const int m = min(kQeTile, c1 - c), first = lo - c, end = hi - c;
        const bool fresh = held != c;
        if (need && fresh) bring(c, m);
        else __syncthreads();                        // the marks are no longer read
#pragma unroll 4
        for (int i = 4 * tid; i < m; i += 4 * kQeThreads) {
            uint32_t keep = 0, tie = 0;
            if (i < end && i + 4 > first && need) {
                uint32_t k[4];
                keys(k, i, fresh);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    keep |= (uint32_t)(k[e] > prefix) << e;
                    tie |= (uint32_t)(k[e] == prefix) << e;
                }
            }
            if (i < first || i + 4 > end || i + 4 > m) {         // slots that stay whatever their weight, or are none
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int j = i + e;
                    if (j < m && j >= first && j < end) continue;
                    keep = (keep & ~(1u << e)) | (uint32_t)(j < m) << e;
                    tie &= ~(1u << e);
                }
            }
            reinterpret_cast<uint8_t *>(sm.sums)[i >> 2] = (uint8_t)(keep | tie << 4);
        }
        if (need) held = c;
        __syncthreads();
    };
    // keep and tie bits of the thread's 32 slots of a tile
    auto marked = [&](int c, uint32_t *keep, uint32_t *tie) {
        uint2 w = make_uint2(0, 0);
        const int m = min(kQeTile, c1 - c);
        if (32 * tid < m) w = reinterpret_cast<const uint2 *>(sm.sums)[tid];
        auto nibbles = [](uint32_t x) { x &= 0x0f0f0f0fu; x = (x | x >> 4) & 0x00ff00ffu; return (x | x >> 8) & 0xffffu; };
        *keep = nibbles(w.x) | nibbles(w.y) << 16;
        *tie = nibbles(w.x >> 4) | nibbles(w.y >> 4) << 16;
        const uint32_t there = 32 * tid + 32 <= m ? 0xffffffffu : 32 * tid < m ? (1u << (m & 31)) - 1 : 0u;   // marks behind the last slot are old
        *keep &= there;
        *tie &= there;
    };
    const bool one = c1 - c0 <= kQeTile;             // one tile: marked once

    // kept and tied slots of this CTA, and of those before it
    uint32_t before = 0, ties_before = 0;
    if (!ALONE) {
        uint32_t kept = 0, ties = 0;
        for (int c = c0; c < c1; c += kQeTile) {
            uint32_t keep, tie;
            mark(c);
            marked(c, &keep, &tie);
            kept += __popc(keep);
            ties += __popc(tie);
        }
        if (tid < 2) sm.count[tid] = 0;
        __syncthreads();
        kept = __reduce_add_sync(kFull, kept);
        ties = __reduce_add_sync(kFull, ties);
        if (lane == 0) {
            atomicAdd(&sm.count[0], kept);
            atomicAdd(&sm.count[1], ties);
        }
        cluster.sync();
        for (int w = 0; w < rank; w++) {
            const uint32_t *o = cluster.map_shared_rank(sm.count, w);
            before += o[0];
            ties_before += o[1];
        }
        before += min(ties_before, left);            // ties that stay are the lowest
        cluster.barrier_arrive();                    // the other CTAs' memory has been read
    }
    for (int c = c0; c < c1; c += kQeTile) {
        if (ALONE || !one) mark(c);
        uint32_t keep, tie, total;
        marked(c, &keep, &tie);
        // slots that stay in any case (upper half) and ties before the thread's
        const uint32_t scan = block_excl_scan<kQeThreads>(__popc(keep) << 16 | __popc(tie), sm.ws, &total);
        uint32_t rest = ties_before + (scan & 0xffffu), at = (scan >> 16) + min(rest, left) - min(ties_before, left);
        const int moved = (int)((total >> 16) + min(ties_before + (total & 0xffffu), left) - min(ties_before, left));
        ties_before += total & 0xffffu;
        for (; tie && rest < left; tie &= tie - 1, rest++) keep |= tie & -tie;
        for (; keep; keep &= keep - 1) sm.list[at++] = (uint16_t)(32 * tid + __ffs(keep) - 1);
        __syncthreads();
        if (ALONE) {                     // each of the pair's CTAs moves a share
            const int share = (moved + gridDim.x - 1) / gridDim.x, j = min(moved, (int)blockIdx.x * share);
            move_rows(a, p, c, sm.list + j, min(share, moved - j), before + j);
        } else {
            move_rows(a, p, c, sm.list, moved, before);
        }
        before += moved;
        __syncthreads();
    }
    const int64_t kept = all ? n : a.budget;
    if (a.keep)
        for (int64_t o = kept + (int)blockIdx.x * kQeThreads + tid; o < a.budget; o += (int64_t)gridDim.x * kQeThreads)
            a.keep[p * a.budget + o] = -1;
    if (blockIdx.x == 0 && tid == 0) a.dst.lens[p] = (int32_t)kept;
    if (late && tid == 0 && a.src.status && atomicCAS(a.src.status, 0, (int)PK_ERR_TIMEOUT) == 0) a.src.status[1] = p;
    if (!ALONE) cluster.barrier_wait();              // and this CTA's by the others
}

cudaError_t launch_quant_evict(const QuantEvictArgs &a, cudaStream_t s)
{
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static std::atomic<int> done[2][kMaxDevices];
    const bool alone = a.src.n_cap <= kQeTile;
    auto kern = alone ? k_quant_evict<true> : k_quant_evict<false>;
    e = dyn_smem_limit(kern, (int)sizeof(QeSmem), done[alone]);
    if (e != cudaSuccess) return e;
    // CTAs per pair: as many as hold its slots in shared memory, and more while there is room for all at once and 128
    // slots for each
    int c = 1;
    while (c < kQeMaxCluster && ((!alone && a.src.n_cap > (int64_t)c * kQeTile) ||
                                 (2 * c * a.src.bh <= 2 * sms && a.src.n_cap >= 2 * c * 128)))
        c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c, a.src.bh);
    cfg.blockDim = dim3(kQeThreads);
    cfg.dynamicSmemBytes = sizeof(QeSmem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = alone ? attr + 1 : attr;
    cfg.numAttrs = alone ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace pk
