// k_quant_evict.cu -- eviction from the 4-bit KV cache by accumulated weight.
//
// Of a pair's keys the first `sink` and the last `recent` stay; of the others
// the heaviest, ties to the lower slots.  A radix select over the ordered bits
// of acc (digits of 11, 10 and 11 bits) gives the threshold weight; the kept
// slots are listed in order and their rows moved.  Instructions bound the
// select, so every step takes 4 slots a lane.  The result does not depend on
// how slots are split.
//
// k_quant_evict, up to kQeTile slots a pair: they stay in a CTA's shared
// memory.  Each of a pair's CTAs selects for itself and moves a share of the
// rows: reading acc again costs less than cluster barriers (64 pairs of 1600
// keys: 24 us for 29).
// k_quant_select, k_quant_gather, longer pairs: a cluster selects, each CTA a
// run of slots; histograms are joined through distributed shared memory, and a
// CTA's own counts above the threshold give its places.  A run is read twice
// (from L2 the second time): for the first digit, and to mark the slots above
// it and put aside those that agree with it, which alone the other digits need
// (64 pairs of 131072 keys to 4096: 38 us, 55 with a pass for each digit and
// one for the marks).  Runs that are too long, or have too many that agree, do
// take those passes.  The list of kept slots goes to `keep`, or to dst's acc
// (whose weights the gather writes in their place), and a second kernel moves
// the rows, all SMs' memory pipes full.  With neither, the cluster moves them
// itself.
#include <cooperative_groups.h>

#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace cg = cooperative_groups;

namespace pk {

constexpr int kQeThreads = 512;
constexpr int kQeBins = 2048;
constexpr int kQeTile = 16384;           // slots in shared memory: two CTAs to an SM
constexpr int kQgThreads = 256;          // gather
constexpr int kQeMaxCluster = 8;

struct QeSmem {
    uint32_t key[kQeTile];               // weights as they come, then their keys
    uint16_t list[kQeTile];              // kept slots
    uint32_t hist[kQeBins];
    uint8_t marks[kQeTile / 4];          // of 4 slots: bits 0..3 those that stay, 4..7 those that tie
    uint32_t ws[kQeThreads / 32 + 1];
    uint32_t digit, left, whole;
    unsigned long long bar;              // bulk copies of the weights
};
static_assert(kQeTile == 32 * kQeThreads, "a thread has one group of the slots");

// The select's CTAs: of 256 threads, 4 to an SM, where there are many pairs; of
// 1024 where each has an SM for itself: four times the loads in flight, and
// room for the marks of a longer run (4 pairs of 1048576 keys: 56 us
// for 122).
constexpr int kQsCopies = 4;             // of the first digit's counts: weights crowd in few bins (one copy: 66 us, four: 50)
constexpr int kQsMany = 256, kQsFew = 1024;
template <int NT>
struct QsState {
    uint32_t ws[NT / 32 + 1];
    uint32_t digit, left, whole;
    uint32_t count[2];                   // kept and tied slots of this CTA
    uint32_t all[kQeMaxCluster];         // `cands` of the cluster's CTAs
    uint32_t ahead[2];                   // of the CTAs before: slots put aside that stay, and that tie
    uint32_t cands;                      // slots put aside, in any order: they agree with the threshold in the first digit
};
template <int NT>
struct QsSmem : QsState<NT> {
    static constexpr int kMarked = 262144, kCands = 6144;        // slots of a run that are marked in the second pass; put aside
    uint32_t sums[kQeBins];              // all CTAs' counts
    uint32_t hist[kQsCopies][kQeBins];   // this CTA's counts
    uint32_t key[kCands];                // of the slots put aside
    uint32_t cand[kCands];
    alignas(16) uint8_t mark[kMarked / 4];
    uint16_t list[32 * NT];              // kept slots of 32 a thread
    __device__ uint32_t *keys() { return key; }
    __device__ uint8_t *marks() { return mark; }
    __device__ uint16_t *chunk() { return list; }
};
template <>
struct QsSmem<kQsMany> : QsState<kQsMany> {
    static constexpr int kMarked = 32768, kCands = 3584;
    alignas(16) uint32_t sums[kQeBins];  // at the end, with hist[0], the list: other CTAs no longer read them
    uint32_t hist[kQsCopies][kQeBins];   // 1, 2: later the keys, 3: marks
    uint16_t cand[kCands];
    __device__ uint32_t *keys() { return hist[1]; }
    __device__ uint8_t *marks() { return reinterpret_cast<uint8_t *>(hist[3]); }
    __device__ uint16_t *chunk() { return reinterpret_cast<uint16_t *>(sums); }
};
static_assert(QsSmem<kQsMany>::kMarked / 4 <= kQeBins * 4 && 8 * kQsMany <= kQeBins * 4 && QsSmem<kQsMany>::kCands <= 2 * kQeBins &&
              2 * 32 * kQsMany <= 2 * kQeBins * 4, "marks, keys and the list fit where they are put");
static_assert(sizeof(QsSmem<kQsMany>) <= 48 * 1024 && sizeof(QsSmem<kQsFew>) <= 227 * 1024, "4 CTAs to an SM, and one");
constexpr int kQsShared = 8192;          // put aside by all CTAs, up to which each takes all of them itself

// digit d of the select: its place, its bins, and the bits above it
struct Digit {
    int shift, bins;
    uint32_t above;
};
__device__ __forceinline__ Digit digit_of(int d)
{
    return d == 0 ? Digit{21, 2048, 0u} : d == 1 ? Digit{11, 1024, 0xffe00000u} : Digit{0, 2048, 0xfffff800u};
}

// ordered bits of a weight; NaN sorts below everything
__device__ __forceinline__ uint32_t weight_key(float x)
{
    return x != x ? 0u : ord_f32(x + 0.0f);
}

// The weight of a key (not NaN's).
__device__ __forceinline__ float key_weight(uint32_t k) { return unord_f32(k); }

// The largest weight whose key agrees with `prefix` in the bits `above`.  No
// weight has the key of -0, 0x7fffffff: as a float it would take in the zeros,
// which belong to the next digit.
__device__ __forceinline__ float top_weight(uint32_t prefix, uint32_t above)
{
    const uint32_t k = prefix | ~above;
    return key_weight(k == 0x7fffffffu ? k - 1 : min(k, 0xff800000u));       // up to infinity
}

// The bin of the left-th largest key by the counts `sums`: *digit, in *rank its
// rank within the bin, and in *whole whether that is the bin's last; over a CTA
// of NT threads.
template <int NT>
__device__ __forceinline__ void find_digit(const uint32_t *sums, int bins, uint32_t *ws, uint32_t left, uint32_t *digit, uint32_t *rank,
                                           uint32_t *whole)
{
    constexpr int kMost = kQeBins / NT;
    const int per = bins / NT, tid = threadIdx.x;
    uint32_t mine[kMost], total = 0, sum;
#pragma unroll
    for (int e = 0; e < kMost; e++) {
        mine[e] = e < per ? sums[per * tid + e] : 0u;
        total += mine[e];
    }
    uint32_t over = block_excl_scan<NT>(total, ws, &sum);
    over = sum - over - total;           // keys in the bins above the thread's
#pragma unroll
    for (int e = kMost - 1; e >= 0; e--) {
        if (over < left && over + mine[e] >= left) {
            *digit = per * tid + e;
            *rank = left - over;
            *whole = left - over == mine[e];
        }
        over += mine[e];
    }
    __syncthreads();
}

// After the second digit: where the whole bin stays the third is not needed, the
// threshold is just below the bin and nothing ties (64 pairs of 1600 keys: 21.7
// us for 22.5).  Not next to zero, whose two signs are one weight.
__device__ __forceinline__ bool bin_stays(uint32_t whole, uint32_t prefix) { return whole && prefix > 0x80000000u; }

// Up to 32 rows to slots o .. o + m - 1 of dst by a warp, lane j < m with the
// source slot of row j: 16 bytes a lane, all loads in flight.
__device__ __forceinline__ void move_rows(const QuantEvictArgs &a, int p, int slot, int m, int64_t o0, bool write_keep)
{
    const int lane = threadIdx.x & 31;
    const uint8_t *src = a.src.blocks + (int64_t)p * (a.src.n_cap / kQKeys) * kQBlock;
    uint8_t *dst = a.dst.blocks + (int64_t)p * (a.dst.n_cap / kQKeys) * kQBlock;
    uint4 kc[4], vc[4];
    uint2 ks = make_uint2(0, 0), vs = ks;
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {        // rows 8i + lane / 4, quarter lane % 4
        const int j = 8 * i + (lane >> 2), x = __shfl_sync(kFull, slot, j);
        if (j < m) {
            const uint8_t *b = src + (int64_t)(x / kQKeys) * kQBlock + x % kQKeys * kQRow;
            kc[i] = __ldcs(reinterpret_cast<const uint4 *>(b) + (lane & 3));
            // chunk places of V differ by the turn of the slot: taken in the order of slots with no turn
            vc[i] = __ldcs(reinterpret_cast<const uint4 *>(b + kQOffV) + ((lane & 3) ^ (v_turn(x) >> 1)));
        }
    }
    if (lane < m) {
        const uint8_t *b = src + (int64_t)(slot / kQKeys) * kQBlock;
        ks = *reinterpret_cast<const uint2 *>(b + kQOffKs + 8 * (slot % kQKeys));
        vs = *reinterpret_cast<const uint2 *>(b + kQOffVs + 8 * (slot % kQKeys));
        if (a.dst.acc) w = a.src.acc[(int64_t)p * a.src.n_cap + slot];
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int j = 8 * i + (lane >> 2);
        if (j < m) {
            const int64_t o = o0 + j;
            const int y = (int)(o % kQKeys);
            uint8_t *b = dst + o / kQKeys * kQBlock + y * kQRow;
            reinterpret_cast<uint4 *>(b)[lane & 3] = kc[i];
            reinterpret_cast<uint4 *>(b + kQOffV)[(lane & 3) ^ (v_turn(y) >> 1)] = vc[i];
        }
    }
    if (lane < m) {
        const int64_t o = o0 + lane;
        uint8_t *b = dst + o / kQKeys * kQBlock;
        *reinterpret_cast<uint2 *>(b + kQOffKs + 8 * (o % kQKeys)) = ks;
        *reinterpret_cast<uint2 *>(b + kQOffVs + 8 * (o % kQKeys)) = vs;
        if (a.dst.acc) a.dst.acc[p * a.dst.n_cap + o] = w;
        if (write_keep && a.keep) a.keep[p * a.budget + o] = slot;
    }
}

// Slots of a pair: all of them stay, or `need` of the contested [lo, hi) and the others.
struct Contest {
    int n, lo, hi;
    uint32_t need;
};
__device__ __forceinline__ Contest contest(const QuantEvictArgs &a, int p)
{
    const int n = quant_len(a.src, p);
    if (n <= a.budget) return Contest{n, n, n, 0u};
    return Contest{n, (int)a.sink, n - (int)a.recent, (uint32_t)(a.budget - a.sink - a.recent)};
}

// Marks of 4 slots a byte, bits 0..3 those that stay and 4..7 those that tie:
// the bits of a thread's 32 slots, of which the first `there` are.
__device__ __forceinline__ void marked(const uint8_t *marks, int there, uint32_t *keep, uint32_t *tie)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(marks);
    auto nibbles = [](uint32_t x) { x &= 0x0f0f0f0fu; x = (x | x >> 4) & 0x00ff00ffu; return (x | x >> 8) & 0xffffu; };
    const uint32_t mask = there >= 32 ? 0xffffffffu : there > 0 ? (1u << there) - 1 : 0u;       // marks behind are old
    *keep = (nibbles(w.x) | nibbles(w.y) << 16) & mask;
    *tie = (nibbles(w.x >> 4) | nibbles(w.y >> 4) << 16) & mask;
}

// What is the same in both ways: the length, the end of the list, the check.
__device__ __forceinline__ void finish(const QuantEvictArgs &a, int p, int n, int threads)
{
    const int64_t kept = min((int64_t)n, a.budget);
    if (a.keep)
        for (int64_t o = kept + (int)blockIdx.x * threads + (int)threadIdx.x; o < a.budget; o += (int64_t)gridDim.x * threads)
            a.keep[p * a.budget + o] = -1;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.dst.lens[p] = (int32_t)kept;
        if (quant_len_bad(a.src, p)) quant_devchk(a.src.status, p);
    }
}

__global__ void __launch_bounds__(kQeThreads, 2) k_quant_evict(QuantEvictArgs a)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    QeSmem &sm = *reinterpret_cast<QeSmem *>(smem_raw);
    const int p = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&sm.bar);
    if (tid == 0) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
    pdl_wait();
    const Contest q = contest(a, p);
    const int n = q.n;
    const float *acc = a.src.acc + (int64_t)p * a.src.n_cap;
    uint32_t prefix = 0, left = q.need;
    bool late = false;
    if (q.need) {
        // weights by bulk copies where they are aligned: all bytes on their way at once, and no register waits for them
        const int bulk = (uintptr_t)acc % 16 == 0 ? n / 4 * 4 : 0;
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncthreads();
        if (bulk && tid == 0) {
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(4 * bulk) : "memory");
            for (int i = 0; i < bulk; i += 4096)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(sm.key + i)),
                             "l"(acc + i), "r"(4 * min(4096, bulk - i)), "r"(bar)
                             : "memory");
        }
        for (int i = bulk + tid; i < n; i += kQeThreads) sm.key[i] = __float_as_uint(acc[i]);
        bool done = !bulk;
        for (int i = 0; i < (1 << 22) && !done; i++) {           // bounded
            uint32_t ok;
            asm volatile(
                "{\n.reg .pred p;\n"
                "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0;\n"
                "selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(ok)
                : "r"(bar)
                : "memory");
            done = ok;
        }
        late = !done;
#pragma unroll 1
        for (int d = 0; d < 3; d++) {
            const Digit g = digit_of(d);
            for (int i = tid; i < g.bins; i += kQeThreads) sm.hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int i = 4 * tid; i < n; i += 4 * kQeThreads) {
                const uint4 v = *reinterpret_cast<const uint4 *>(sm.key + i);
                uint32_t k[4] = {v.x, v.y, v.z, v.w};
                if (d == 0) {
#pragma unroll
                    for (int e = 0; e < 4; e++) k[e] = weight_key(__uint_as_float(k[e]));
                    *reinterpret_cast<uint4 *>(sm.key + i) = make_uint4(k[0], k[1], k[2], k[3]);
                }
                bool any = d == 0;                               // few agree with the digits before
#pragma unroll
                for (int e = 0; e < 4; e++) any |= (k[e] & g.above) == prefix;
                if (!any) continue;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (i + e >= q.lo && i + e < q.hi && (k[e] & g.above) == prefix)
                        atomicAdd(&sm.hist[(k[e] >> g.shift) & (g.bins - 1)], 1u);
            }
            __syncthreads();
            find_digit<kQeThreads>(sm.hist, g.bins, sm.ws, left, &sm.digit, &sm.left, &sm.whole);
            prefix |= sm.digit << g.shift;
            left = sm.left;
            const bool stays = d == 1 && bin_stays(sm.whole, prefix);
            __syncthreads();
            if (stays) {
                prefix--;
                left = 0;
                break;
            }
        }
    }
    for (int i = 4 * tid; i < n; i += 4 * kQeThreads) {
        uint32_t keep = 0, tie = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int j = i + e;
            if (j >= n) continue;
            const bool in = j >= q.lo && j < q.hi;
            const uint32_t k = in && q.need ? sm.key[j] : 0u;
            keep |= (uint32_t)(!in || (q.need && k > prefix)) << e;
            tie |= (uint32_t)(in && q.need && k == prefix) << e;
        }
        sm.marks[i >> 2] = (uint8_t)(keep | tie << 4);
    }
    __syncthreads();
    uint32_t keep, tie, total;
    marked(sm.marks + 8 * tid, n - 32 * tid, &keep, &tie);
    // slots that stay in any case (upper half) and ties before the thread's; ties that stay are the lowest
    const uint32_t scan = block_excl_scan<kQeThreads>(__popc(keep) << 16 | __popc(tie), sm.ws, &total);
    uint32_t rest = scan & 0xffffu, at = (scan >> 16) + min(rest, left);
    const int kept = (int)((total >> 16) + min(total & 0xffffu, left));
    for (; tie && rest < left; tie &= tie - 1, rest++) keep |= tie & -tie;
    for (; keep; keep &= keep - 1) sm.list[at++] = (uint16_t)(32 * tid + __ffs(keep) - 1);
    __syncthreads();
    const int share = (kept + (int)gridDim.x - 1) / (int)gridDim.x, j0 = min(kept, (int)blockIdx.x * share), j1 = min(kept, j0 + share);
    for (int j = j0 + 32 * warp; j < j1; j += kQeThreads) {
        const int m = min(32, j1 - j);
        move_rows(a, p, lane < m ? (int)sm.list[j + lane] : 0, m, j, true);
    }
    finish(a, p, n, kQeThreads);
    if (late && tid == 0) quant_late(a.src.status, p);
}

// where a long pair's kept slots are listed: null where the select kernel moves the rows
__device__ __forceinline__ int *kept_list(const QuantEvictArgs &a, int p)
{
    return a.keep ? a.keep + p * a.budget : a.dst.acc ? reinterpret_cast<int *>(a.dst.acc + p * a.dst.n_cap) : nullptr;
}

template <int NT>
__device__ __forceinline__ void quant_select(const QuantEvictArgs &a, QsSmem<NT> &sm)
{
    using Smem = QsSmem<NT>;
    cg::cluster_group cluster = cg::this_cluster();
    const int p = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    pdl_wait();
    const Contest q = contest(a, p);
    const float *acc = a.src.acc + (int64_t)p * a.src.n_cap;
    const bool vec = (uintptr_t)acc % 16 == 0;       // n_cap is a multiple of 32: the same for every pair
    const int run = (int)((((int64_t)q.n + ranks - 1) / ranks + 3) / 4 * 4);
    const int c0 = (int)min((int64_t)q.n, (int64_t)rank * run), c1 = min(q.n, c0 + run);
    // weights of slots i .. i + 3 (behind c1: NaN)
    auto weights = [&](float x[4], int i) {
        if (vec && i + 4 <= c1) {
            const float4 v = *reinterpret_cast<const float4 *>(acc + i);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = i + e < c1 ? acc[i + e] : __uint_as_float(0x7fffffffu);
        }
    };

    // f(weights, i) for the slots i .. i + 3 of [from, stop), 4 loads in flight
    auto each = [&](int from, int stop, auto &&f) {
        int i = from + 4 * tid;
        for (; vec && i + 12 * NT + 4 <= stop; i += 16 * NT) {
            float4 v[4];
#pragma unroll
            for (int h = 0; h < 4; h++) v[h] = *reinterpret_cast<const float4 *>(acc + i + 4 * h * NT);
#pragma unroll
            for (int h = 0; h < 4; h++) {
                const float x[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
                f(x, i + 4 * h * NT);
            }
        }
        for (; i < stop; i += 4 * NT) {
            float x[4];
            weights(x, i);
            f(x, i);
        }
    };

    uint8_t *marks = sm.marks();
    uint32_t *cand_key = sm.keys();
    const bool once = run <= Smem::kMarked;
    bool marks_done = false, alone = false;
    const uint32_t others = (uint32_t)(c1 - c0 - max(0, min(c1, q.hi) - max(c0, q.lo)));       // not contested
    if (tid == 0) {
        sm.cands = sm.ahead[0] = sm.ahead[1] = 0;
        sm.count[0] = others;
    }
    // f(key) for the keys that the first `upto` CTAs have put aside
    auto each_cand = [&](int upto, auto &&f) {
        uint32_t most = 0;
        for (int w = 0; w < upto; w++) most = max(most, sm.all[w]);
        for (uint32_t i = tid; i < most; i += NT) {
            uint32_t k[kQeMaxCluster];
#pragma unroll
            for (int w = 0; w < kQeMaxCluster; w++) k[w] = w < upto && i < sm.all[w] ? cluster.map_shared_rank(cand_key, w)[i] : 0u;
#pragma unroll
            for (int w = 0; w < kQeMaxCluster; w++)
                if (w < upto && i < sm.all[w]) f(k[w]);
        }
    };
    // threshold key, and how many of the keys equal to it stay; own: this CTA's contested keys above it
    uint32_t prefix = 0, left = q.need, own = 0, ties = 0;
    if (q.need) {
#pragma unroll 1
        for (int d = 0; d < 3; d++) {
            const Digit g = digit_of(d);
            const int copies = d == 0 ? kQsCopies : 1;
            for (int i = tid; i < copies * kQeBins; i += NT) sm.hist[0][i] = 0;
            __syncthreads();
            // the contested part of the run, from a multiple of 4 on
            const int first = max(c0, q.lo), end = min(c1, q.hi);
            // keys that agree with the digits before are a range of weights (the first digit 0: NaN alone)
            const bool nan = d > 0 && (prefix >> 21) == 0;
            const float low = d == 0 || nan ? 0.0f : key_weight(max(prefix, 0x007fffffu));                 // -inf
            const float high = d == 0 || nan ? 0.0f : top_weight(prefix, g.above);
            uint32_t *hist = sm.hist[d == 0 ? lane & (kQsCopies - 1) : 0];
            auto count = [&](const float x[4], int i) {
                if (d > 0 && !nan) {                 // few
                    bool any = false;
#pragma unroll
                    for (int e = 0; e < 4; e++) any |= x[e] >= low && x[e] <= high;
                    if (!any) return;
                }
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const uint32_t k = weight_key(x[e]);
                    if (i + e >= first && i + e < end && (k & g.above) == prefix) atomicAdd(&hist[(k >> g.shift) & (g.bins - 1)], 1u);
                }
            };
            // first digit: of all contested slots
            auto count_first = [&](const float x[4], int i) {
                if (i >= first && i + 4 <= end) {
#pragma unroll
                    for (int e = 0; e < 4; e++) atomicAdd(&hist[weight_key(x[e]) >> 21], 1u);
                } else {
                    count(x, i);
                }
            };
            // second digit: also marks the slots above the first, and puts aside those that agree with it
            auto count_and_mark = [&](const float x[4], int i) {
                uint32_t above = 0, from = 0, in = 15;
                if (i < first || i + 4 > end) {
                    in = 0;
#pragma unroll
                    for (int e = 0; e < 4; e++) in |= (uint32_t)(i + e >= first && i + e < end) << e;
                }
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    above |= (uint32_t)(nan ? x[e] == x[e] : x[e] > high) << e;
                    from |= (uint32_t)(nan || x[e] >= low) << e;
                }
                marks[(i - c0) >> 2] = (uint8_t)((above | ~in) & 15u);
                for (uint32_t c = from & ~above & in; c; c &= c - 1) {
                    const int e = __ffs(c) - 1;
                    const uint32_t k = weight_key(e == 0 ? x[0] : e == 1 ? x[1] : e == 2 ? x[2] : x[3]), at = atomicAdd(&sm.cands, 1u);
                    atomicAdd(&hist[(k >> g.shift) & (g.bins - 1)], 1u);
                    if (at < Smem::kCands) {
                        cand_key[at] = k;
                        sm.cand[at] = i + e - c0;
                    }
                }
            };
            if (d == 0) {
                each(first / 4 * 4, end, count_first);
            } else if (d == 1 && once) {
                each(c0, c1, count_and_mark);
            } else if (marks_done) {
                for (int i = tid; i < (int)sm.cands; i += NT)
                    if ((cand_key[i] & g.above) == prefix) atomicAdd(&hist[(cand_key[i] >> g.shift) & (g.bins - 1)], 1u);
            } else {
                each(first / 4 * 4, end, count);
            }
            if (d == 0) {
                __syncthreads();
                for (int i = tid; i < kQeBins; i += NT) {
                    uint32_t v = 0;
#pragma unroll
                    for (int w = 0; w < kQsCopies; w++) v += sm.hist[w][i];
                    sm.hist[0][i] = v;
                }
            }
            if (d == 1 && once) {
                const uint32_t above = __reduce_add_sync(kFull, own);
                if (lane == 0) atomicAdd(&sm.count[0], above);
            }
            cluster.sync();
            if (d == 1 && once) {
                if (tid < ranks) sm.all[tid] = *cluster.map_shared_rank(&sm.cands, tid);
                __syncthreads();
                uint32_t total = 0, most = 0;
                for (int w = 0; w < ranks; w++) total += sm.all[w], most = max(most, sm.all[w]);
                alone = most <= Smem::kCands && total <= kQsShared;
            }
            if (alone) {                 // the other digits without the other CTAs' help
                marks_done = true;
#pragma unroll 1
                for (int e = 1; e < 3; e++) {
                    const Digit h = digit_of(e);
                    for (int i = tid; i < h.bins; i += NT) sm.sums[i] = 0;
                    __syncthreads();
                    each_cand(ranks, [&](uint32_t k) {
                        if ((k & h.above) == prefix) atomicAdd(&sm.sums[(k >> h.shift) & (h.bins - 1)], 1u);
                    });
                    __syncthreads();
                    find_digit<NT>(sm.sums, h.bins, sm.ws, left, &sm.digit, &sm.left, &sm.whole);
                    prefix |= sm.digit << h.shift;
                    left = sm.left;
                    const bool stays = e == 1 && bin_stays(sm.whole, prefix);
                    __syncthreads();
                    if (stays) {
                        prefix--;
                        left = 0;
                        break;
                    }
                }
                break;
            }
            // each CTA joins the counts of its share of the bins and gives all the sums
            const int share = g.bins / ranks;
            for (int i = tid; i < share; i += NT) {
                uint32_t x[kQeMaxCluster], v = 0;
#pragma unroll
                for (int w = 0; w < kQeMaxCluster; w++) x[w] = w < ranks ? cluster.map_shared_rank(sm.hist[0], w)[rank * share + i] : 0u;
#pragma unroll
                for (int w = 0; w < kQeMaxCluster; w++) v += x[w];
#pragma unroll
                for (int w = 0; w < kQeMaxCluster; w++)
                    if (w < ranks) cluster.map_shared_rank(sm.sums, w)[rank * share + i] = v;
            }
            cluster.sync();
            find_digit<NT>(sm.sums, g.bins, sm.ws, left, &sm.digit, &sm.left, &sm.whole);
            const uint32_t digit = sm.digit;
            prefix |= digit << g.shift;
            left = sm.left;
            const bool stays = d == 1 && bin_stays(sm.whole, prefix);
            for (int i = tid; i < g.bins; i += NT)
                if (i + (int)stays > (int)digit) own += sm.hist[0][i];
            if (d == 2) ties = sm.hist[0][digit];
            if (d == 1) marks_done = once && sm.cands <= Smem::kCands;
            __syncthreads();
            if (stays) {
                prefix--;
                left = 0;
                break;
            }
        }
        if (marks_done)                  // the other slots that stay or tie
            for (int i = tid; i < (int)sm.cands; i += NT) {
                const uint32_t k = cand_key[i], j = sm.cand[i];
                if (k >= prefix) atomicOr(reinterpret_cast<uint32_t *>(marks) + (j >> 4), 1u << (8 * (j >> 2 & 3) + (j & 3) + (k == prefix ? 4 : 0)));
            }
    }
    // kept slots before this CTA's
    uint32_t before = 0, ties_before = 0;
    if (alone) {
        uint32_t above = 0, equal = 0;
        each_cand(rank, [&](uint32_t k) { above += k > prefix, equal += k == prefix; });
        above = __reduce_add_sync(kFull, above);
        equal = __reduce_add_sync(kFull, equal);
        if (lane == 0) {
            atomicAdd(&sm.ahead[0], above);
            atomicAdd(&sm.ahead[1], equal);
        }
        for (int w = 0; w < rank; w++) before += *cluster.map_shared_rank(sm.count, w);
        __syncthreads();
        before += sm.ahead[0];
        ties_before = sm.ahead[1];
        before += min(ties_before, left);            // ties that stay are the lowest
        cluster.barrier_arrive();                    // the other CTAs' memory has been read
    } else {
        own = __reduce_add_sync(kFull, own);
        if (tid == 0) {
            sm.count[0] = others;
            sm.count[1] = ties;
        }
        __syncthreads();
        if (lane == 0) atomicAdd(&sm.count[0], own);
        cluster.sync();
        for (int w = 0; w < rank; w++) {
            const uint32_t *o = cluster.map_shared_rank(sm.count, w);
            before += o[0];
            ties_before += o[1];
        }
        before += min(ties_before, left);
        cluster.barrier_arrive();
    }
    int *list = kept_list(a, p);
    uint16_t *chunk = sm.chunk();
    const bool nan = prefix == 0;                    // the threshold is NaN: all others are above it
    const float limit = nan ? 0.0f : key_weight(prefix);
    for (int c = c0; c < c1; c += 32 * NT) {
        auto mark = [&](const float x[4], int i) {
            uint32_t keep = 0, tie = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const bool in = i + e >= q.lo && i + e < q.hi;
                const bool above = nan ? x[e] == x[e] : x[e] > limit, equal = nan ? x[e] != x[e] : x[e] == limit;
                keep |= (uint32_t)(!in || (q.need && above)) << e;
                tie |= (uint32_t)(in && q.need && equal) << e;
            }
            marks[(i - c) >> 2] = (uint8_t)(keep | tie << 4);
        };
        const int stop = min(c1, c + 32 * NT);
        if (!marks_done) each(c, stop, mark);
        __syncthreads();
        uint32_t keep, tie, total;
        const int i0 = c + 32 * tid;
        marked(marks + (marks_done ? (c - c0) / 4 : 0) + 8 * tid, stop - i0, &keep, &tie);
        const uint32_t scan = block_excl_scan<NT>(__popc(keep) << 16 | __popc(tie), sm.ws, &total);
        uint32_t rest = ties_before + (scan & 0xffffu), at = (scan >> 16) + min(rest, left) - min(ties_before, left);
        const int kept = (int)((total >> 16) + min(ties_before + (total & 0xffffu), left) - min(ties_before, left));
        ties_before += total & 0xffffu;
        for (; tie && rest < left; tie &= tie - 1, rest++) keep |= tie & -tie;
        if (list) {
            for (; keep; keep &= keep - 1) list[before + at++] = i0 + __ffs(keep) - 1;
        } else {
            for (; keep; keep &= keep - 1) chunk[at++] = (uint16_t)(32 * tid + __ffs(keep) - 1);
            __syncthreads();
            for (int j = 32 * warp; j < kept; j += NT) {
                const int m = min(32, kept - j);
                move_rows(a, p, lane < m ? c + chunk[j + lane] : 0, m, before + j, false);
            }
        }
        __syncthreads();                             // the marks and the list have been read
        before += kept;
    }
    finish(a, p, q.n, NT);
    cluster.barrier_wait();                          // and this CTA's by the others
}

__global__ void __launch_bounds__(kQsMany, 4) k_quant_select(QuantEvictArgs a)
{
    __shared__ QsSmem<kQsMany> sm;
    quant_select(a, sm);
}

__global__ void __launch_bounds__(kQsFew, 1) k_quant_select_few(QuantEvictArgs a)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    quant_select(a, *reinterpret_cast<QsSmem<kQsFew> *>(smem_raw));
}

// Rows of the listed slots, a warp 32 of them.
__global__ void __launch_bounds__(kQgThreads) k_quant_gather(QuantEvictArgs a)
{
    const int p = blockIdx.y, lane = threadIdx.x & 31;
    pdl_wait();
    const int kept = (int)min((int64_t)quant_len(a.src, p), a.budget);
    const int *list = kept_list(a, p);
    const int64_t j = (int64_t)blockIdx.x * kQgThreads + (threadIdx.x & ~31);
    if (j >= kept) return;
    const int m = min(32, kept - (int)j);
    move_rows(a, p, lane < m ? list[j + lane] : 0, m, j, false);
}

cudaError_t launch_quant_evict(const QuantEvictArgs &a, cudaStream_t s)
{
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int c = 1;                           // CTAs per pair
    if (a.src.n_cap <= kQeTile) {
        static std::atomic<int> done[kMaxDevices];
        e = dyn_smem_limit(k_quant_evict, (int)sizeof(QeSmem), done);
        if (e != cudaSuccess) return e;
        // more while there is room for all at once and 128 slots for each
        while (c < 8 && 2 * c * a.src.bh <= 2 * sms && a.src.n_cap >= 2 * c * 128) c *= 2;
        return launch_pdl(k_quant_evict, dim3(c, a.src.bh), dim3(kQeThreads), sizeof(QeSmem), s, a);
    }
    // more while there is room for all at once and four slots for each thread
    // a cluster of large CTAs needs 8 SMs of one part of the GPU: up to 12 pairs are all there at once (16 pairs of
    // 262144 keys: 64 us for 50); fewer slots than 12 a thread do not pay (1 pair of 40007 keys: 24 us for 22, of 131072
    // 25.7 for 26.4)
    const bool few = 12 * a.src.bh <= sms && a.src.n_cap >= (int64_t)kQeMaxCluster * 12 * kQsFew;
    while (c < kQeMaxCluster && (few || 2 * c * a.src.bh <= 4 * sms) && a.src.n_cap >= 2 * c * 4 * kQsMany) c *= 2;
    const int smem = few ? (int)sizeof(QsSmem<kQsFew>) : 0;
    if (few) {
        static std::atomic<int> done[kMaxDevices];
        e = dyn_smem_limit(k_quant_select_few, smem, done);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c, a.src.bh);
    cfg.blockDim = dim3(few ? kQsFew : kQsMany);
    cfg.dynamicSmemBytes = smem;
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
    e = cudaLaunchKernelEx(&cfg, few ? k_quant_select_few : k_quant_select, a);
    if (e != cudaSuccess || !(a.keep || a.dst.acc)) return e;
    const int64_t most = a.budget < a.src.n_cap ? a.budget : a.src.n_cap;
    return launch_pdl(k_quant_gather, dim3((unsigned)((most + kQgThreads - 1) / kQgThreads), a.src.bh), dim3(kQgThreads), 0, s, a);
}

}  // namespace pk
