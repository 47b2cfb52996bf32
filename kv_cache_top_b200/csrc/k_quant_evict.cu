// k_quant_evict.cu -- eviction from the 4-bit KV cache by accumulated weight.
//
// Of a pair's keys the first `sink` and the last `recent` stay; of the others
// the heaviest, ties to the lower slots.  A cluster of CTAs serves a pair, each
// CTA a run of its slots: a radix select over the ordered bits of acc (three
// digits, the CTAs' histograms joined through distributed shared memory)
// gives the threshold weight, the CTAs' counts of kept keys and ties their
// places, and each CTA moves its own kept rows.
//
// Memory bounds it where rows are long: acc is read once from HBM and three
// more times from L2, kept rows are read and written once.  The order of the
// rows is kept, so the result does not depend on the split.
#include <cooperative_groups.h>

#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace cg = cooperative_groups;

namespace pk {

constexpr int kQeThreads = 512;
constexpr int kQeWarps = kQeThreads / 32;
constexpr int kQeBins = 2048;            // 11, 11 and 10 bits
constexpr int kQeChunk = 4 * kQeThreads; // slots a CTA looks at in one step
constexpr int kQeMaxCluster = 8;

struct QeSmem {
    uint32_t hist[2][kQeBins];           // of the digit in turn: while the CTAs still read one, the next counts
    uint32_t ws[kQeWarps + 1];
    uint32_t digit, left;
    uint32_t count[2];                   // kept and tied slots of this CTA
    int list[kQeChunk];
};

// ordered bits of a weight; NaN sorts below everything
__device__ __forceinline__ uint32_t weight_key(float x)
{
    return x != x ? 0u : ord_f32(x + 0.0f);
}

// slots 4 at a time: the CTA's thread t has slots at + 4t .. + 3 (outside [lo, hi): 0 and not counted)
__device__ __forceinline__ void load_keys(uint32_t k[4], const float *acc, int64_t i, int64_t hi, bool vec)
{
    if (vec && i + 4 <= hi) {
        const float4 v = *reinterpret_cast<const float4 *>(acc + i);
        k[0] = weight_key(v.x), k[1] = weight_key(v.y), k[2] = weight_key(v.z), k[3] = weight_key(v.w);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++) k[e] = i + e < hi ? weight_key(acc[i + e]) : 0u;
    }
}

// Rows src[list[j]] to slots o0 + j, j < count (pair bases), by the CTA's
// warps: 32 rows at a time, 16 bytes a lane.
__device__ __forceinline__ void move_rows(const QuantEvictArgs &a, int p, const int *list, int count, int64_t o0)
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
                const int x = list[j0 + j];
                const uint8_t *b = src + (int64_t)(x / kQKeys) * kQBlock + x % kQKeys * kQRow;
                kc[i] = __ldcs(reinterpret_cast<const uint4 *>(b) + (lane & 3));
                // chunk places of V differ by the turn of the slot: taken in the order of slots with no turn
                vc[i] = __ldcs(reinterpret_cast<const uint4 *>(b + kQOffV) + ((lane & 3) ^ (v_turn(x) >> 1)));
            }
        }
        if (lane < m) {
            slot = list[j0 + lane];
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

__global__ void __launch_bounds__(kQeThreads, 2) k_quant_evict(QuantEvictArgs a)
{
    __shared__ QeSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int p = blockIdx.y, tid = threadIdx.x, rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    pdl_wait();
    const int n = quant_len(a.src, p);
    if (rank == 0 && tid == 0 && quant_len_bad(a.src, p)) quant_devchk(a.src.status, p);
    const float *acc = a.src.acc + (int64_t)p * a.src.n_cap;
    const bool vec = (uintptr_t)acc % 16 == 0;       // n_cap is a multiple of 32: the same for every pair
    const bool all = n <= a.budget;
    const int lo = all ? n : (int)a.sink, hi = all ? n : n - (int)a.recent;   // contested slots
    const uint32_t need = all ? 0u : (uint32_t)(a.budget - a.sink - a.recent);
    // this CTA's slots [c0, c1)
    const int64_t run = ((n + ranks - 1) / ranks + 3) / 4 * 4;
    const int64_t c0 = min((int64_t)n, rank * run), c1 = min((int64_t)n, c0 + run);
    auto contested = [&](int64_t i) { return i >= lo && i < hi; };

    // threshold key: the need-th largest of the contested; left: how many of those equal to it stay
    uint32_t prefix = 0, left = need;
    if (need) {
#pragma unroll
        for (int d = 0; d < 3; d++) {
            const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : 2048;
            const uint32_t above = d == 0 ? 0u : d == 1 ? 0xffe00000u : 0xfffffc00u;
            uint32_t *hist = sm.hist[d & 1];
            for (int i = tid; i < bins; i += kQeThreads) hist[i] = 0;
            __syncthreads();
            for (int64_t c = c0; c < c1; c += kQeChunk) {
                const int64_t i = c + 4 * tid;
                uint32_t k[4];
                load_keys(k, acc, i, c1, vec);
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (i + e < c1 && contested(i + e) && (k[e] & above) == prefix) atomicAdd(&hist[(k[e] >> shift) & (bins - 1)], 1u);
            }
            cluster.sync();
            // all CTAs' counts; thread t has bins [per t, per (t + 1))
            const int per = bins / kQeThreads;
            uint32_t mine[4], total = 0;
            for (int e = 0; e < per; e++) {
                mine[e] = 0;
                for (int w = 0; w < ranks; w++) mine[e] += cluster.map_shared_rank(hist, w)[per * tid + e];
                total += mine[e];
            }
            uint32_t sum;
            uint32_t over = block_excl_scan<kQeThreads>(total, sm.ws, &sum);
            over = sum - over - total;               // keys in the bins above the thread's
            for (int e = per - 1; e >= 0; e--) {
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
    // kept and tied slots of this CTA, and of those before it
    uint32_t before = 0, ties_before = 0;
    {
        uint32_t kept = 0, ties = 0;
        for (int64_t c = c0; c < c1; c += kQeChunk) {
            const int64_t i = c + 4 * tid;
            uint32_t k[4];
            if (need) load_keys(k, acc, i, c1, vec);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (i + e >= c1) continue;
                if (!contested(i + e)) kept++;
                else if (need && k[e] > prefix) kept++;
                else if (need && k[e] == prefix) ties++;
            }
        }
        kept = __reduce_add_sync(kFull, kept);
        ties = __reduce_add_sync(kFull, ties);
        if (tid < 2) sm.count[tid] = 0;
        __syncthreads();
        if ((tid & 31) == 0) {
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
    }
    for (int64_t c = c0; c < c1; c += kQeChunk) {
        const int64_t i = c + 4 * tid;
        uint32_t k[4];
        if (need) load_keys(k, acc, i, c1, vec);
        uint32_t keep = 0, tie = 0;                  // bit e: slot i + e
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if (i + e >= c1) continue;
            if (!contested(i + e) || (need && k[e] > prefix)) keep |= 1u << e;
            else if (need && k[e] == prefix) tie |= 1u << e;
        }
        uint32_t total;
        uint32_t rest = block_excl_scan<kQeThreads>(__popc(tie), sm.ws, &total);
        rest += ties_before;
        ties_before += total;
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (tie >> e & 1) {
                if (rest < left) keep |= 1u << e;
                rest++;
            }
        uint32_t at = block_excl_scan<kQeThreads>(__popc(keep), sm.ws, &total);
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (keep >> e & 1) sm.list[at++] = (int)(i + e);
        __syncthreads();
        move_rows(a, p, sm.list, (int)total, before);
        before += total;
        __syncthreads();
    }
    const int64_t kept = all ? n : a.budget;
    if (a.keep)
        for (int64_t o = kept + rank * kQeThreads + tid; o < a.budget; o += (int64_t)ranks * kQeThreads) a.keep[p * a.budget + o] = -1;
    if (rank == 0 && tid == 0) a.dst.lens[p] = (int32_t)kept;
    cluster.sync();                                  // the CTAs' counts have been read
}

cudaError_t launch_quant_evict(const QuantEvictArgs &a, cudaStream_t s)
{
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // CTAs per pair: about four per SM in all, each with two steps of slots at least
    int c = 1;
    while (c < kQeMaxCluster && 2 * c * a.src.bh <= 4 * sms && a.src.n_cap / (2 * c) >= 2 * kQeChunk) c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c, a.src.bh);
    cfg.blockDim = dim3(kQeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_quant_evict, a);
}

}  // namespace pk
