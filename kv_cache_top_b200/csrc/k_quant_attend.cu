// k_quant_attend.cu -- softmax attention over the 4-bit KV cache.
//
// z_gj = scale <q_g, K_j>, out_g = sum_j softmax(z_g)_j V_j, with an online
// softmax per worker's segment of a pair and a merge of the segments; when
// weights are accumulated, the logits go to the workspace and the merge
// kernel, which knows each head's log-sum, adds the weights to acc.
//
// 144 bytes a key of HBM are the floor (64 pairs of 131072 keys, 4 heads: 184
// us; the kernel takes 267, at the power cap 298 to 306; 8 heads 357).  What
// bounds it is the instructions that make matrix operands of codes and sums of
// digits: 751 warp instructions a block of 32 keys, issue slots 67% full, the
// integer pipe 52%, fp32 46%, matrix 23% (8 heads: 869, 60%, 39%, 43%, 35%).
// Hence bytes and not halves for the logits (292
// us to 275), two fp32 operations an instruction (291 to 276), and 16 warps
// with two blocks each in flight and not 8 or 12 with more (320 and 296).
// Calls of few keys are bound by latency: two launches, a plan, one round of
// blocks and a merge are 8 us.
#include <cuda_fp16.h>

#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace pk {

constexpr int kQaWarps = 16;
constexpr int kQaThreads = 32 * kQaWarps;
constexpr int kQaStages = 2;             // blocks in flight per warp
constexpr int kQaFew = 4;                // warps of a small worker
constexpr int kQaGroups = kQaWarps / kQaFew;
constexpr int kQaCol = kD + 4;           // floats between the columns of a warp's sums in shared memory
constexpr int kQmThreads = 256;          // merge kernel
constexpr int kQmKeys = 2048;            // keys of a merge CTA's part of acc
constexpr int kQmHeads = kQmThreads / kD;      // heads whose outputs are one pass of a merge CTA

struct Place {
    uint32_t pair, first, start, end;    // blocks start .. end - 1 of all; the pair of the first, and that pair's first
};

struct QaSmem {
    uint8_t ring[kQaWarps][kQaStages][kQBlock];
    unsigned long long bar[kQaWarps][kQaStages];
    float4 ks[kQaWarps][kQKeys];         // scales [pair of keys][group][key] of the warp's block, K ...
    float4 vs[kQaWarps][kQKeys];         // ... and V
    float size[kQaWarps][kQKeys];        // exponent of each key's largest V scale
    float m[kQaWarps][8], l[kQaWarps][8];
    float4 qscale[kQaGroups][2][kMaxGroup];      // unit of a logit's part, by groups of channels
    uint32_t ws[kQaWarps + 1];
    float factor[kQaWarps][8];           // of a warp's column in the segment's sums
    uint32_t fits[2][kQaWarps];
    Place place[kQaGroups];
    uint32_t share[kQaGroups];           // blocks a worker takes; by pairs: bit 31 (for the thread that writes it)
    int has[kQaWarps];
    alignas(16) uint32_t q[kQaGroups * 2 * kMaxGroup][4][4][8];  // last: as many as are used; [worker, segment parity, head][digit][group][2 t + h]: bytes of channels 32r + 8t + h + {0, 2, 4, 6}
};
static_assert(offsetof(QaSmem, bar) % 16 == 0 && offsetof(QaSmem, ks) % 16 == 0 && offsetof(QaSmem, vs) % 16 == 0 && offsetof(QaSmem, size) % 16 == 0 &&
              offsetof(QaSmem, qscale) % 16 == 0 && offsetof(QaSmem, q) % 16 == 0, "read 8 and 16 bytes at a time");
static_assert(8 * kQaCol * 4 <= kQBlock, "a warp's sums fit the block that it has consumed");

// blocks a worker of `span` warps takes at least
__host__ __device__ constexpr int min_share(int span) { return span == kQaWarps ? 8 : span; }

__device__ __forceinline__ uint32_t block_count(const QuantCache &c, int p) { return (uint32_t)(quant_len(c, p) + kQKeys - 1) / kQKeys; }

// Block count of all pairs, over the CTA.
__device__ uint32_t count_blocks(const QuantCache &c, uint32_t *s)
{
    uint32_t v = 0;
    for (int p = threadIdx.x; p < c.bh; p += kQaThreads) v += block_count(c, p);
    v = __reduce_add_sync(kFull, v);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kQaWarps; w++) v += s[w];
    __syncthreads();
    return v;
}

// nb / share, rounded up; inv = 1 / share
__device__ __forceinline__ uint32_t ceil_share(uint32_t nb, uint32_t share, float inv)
{
    uint32_t q = (uint32_t)((float)nb * inv);        // off by one at most: quotients stay near the number of workers
    int r = (int)(nb - q * share);
    if (r < 0) q--, r += (int)share;
    if (r >= (int)share) q++, r -= (int)share;
    return q + (r > 0);
}

// Blocks a worker takes of `total` cut evenly.
__device__ __forceinline__ uint32_t even_share(uint32_t total, int workers, int span)
{
    return max((total + (uint32_t)workers - 1) / (uint32_t)workers, (uint32_t)min_share(span));
}

// Up to 32 PER pairs, and no more than workers: a worker takes blocks of one
// pair only, `share` of them, the smallest that does with the workers there
// are, unless that is more than an even share by about a round of the warps,
// what a second merge costs (64 ragged pairs of up to 282 blocks: 35 us by
// pairs, 55 evenly; 64 pairs of 4096 blocks, 2 workers for each and 20 idle:
// 300 and 268).  Else (the result is 0) the pairs' blocks are laid end to end
// and cut evenly.  The share, and the place of `worker` (end 0: no work): warp w
// tries the share w above the even one, and every warp places its worker for
// itself (8 pairs of 32768 keys: 22.6 us; by one warp, with a search and a
// broadcast: 24.3).
template <int PER, int SPAN>
__device__ __forceinline__ uint32_t plan_pairs(const QuantCache &c, int workers, uint32_t worker, int warp, int lane, uint32_t *fits, Place *at)
{
    *at = Place{0u, 0u, 0u, 0u};
    if (c.bh > 32 * PER || c.bh > workers) return 0;
    uint32_t nb[PER], blocks = 0;        // of the pairs PER lane + i
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int p = PER * lane + i;
        nb[i] = p < c.bh ? block_count(c, p) : 0u;
        blocks += nb[i];
    }
    const uint32_t total = __reduce_add_sync(kFull, blocks);
    const uint32_t even = even_share(total, workers, SPAN);
    {
        const uint32_t share = even + warp;
        const float inv = __frcp_rn((float)share);
        uint32_t k = 0;                  // workers at this share
#pragma unroll
        for (int i = 0; i < PER; i++) k += ceil_share(nb[i], share, inv);
        k = __reduce_add_sync(kFull, k);
        if (lane == 0) fits[warp] = warp <= SPAN && k <= (uint32_t)workers;
    }
    __syncthreads();
    const uint32_t ok = __ballot_sync(kFull, lane < kQaWarps && fits[lane & (kQaWarps - 1)]);
    if (ok == 0) return 0;
    const uint32_t share = even + __ffs(ok) - 1;
    const float inv = __frcp_rn((float)share);
    uint32_t k[PER], w = 0, f = blocks;  // sums over the lanes up to this: workers and blocks
#pragma unroll
    for (int i = 0; i < PER; i++) {
        k[i] = ceil_share(nb[i], share, inv);
        w += k[i];
    }
    const uint32_t own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(kFull, w, o), y = __shfl_up_sync(kFull, f, o);
        if (lane >= o) w += x, f += y;
    }
    const uint32_t here = __ballot_sync(kFull, worker < w && worker >= w - own);
    if (here) {                          // the lane that has the worker's pair
        w -= own;
        f -= blocks;
        Place x = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < PER; i++) {
            if (worker >= w && worker - w < k[i]) {
                const uint32_t start = f + (worker - w) * share;
                x = Place{(uint32_t)(PER * lane + i), f, start, min(f + nb[i], start + share)};
            }
            w += k[i];
            f += nb[i];
        }
        const int src = __ffs(here) - 1;
        at->pair = __shfl_sync(kFull, x.pair, src);
        at->first = __shfl_sync(kFull, x.first, src);
        at->start = __shfl_sync(kFull, x.start, src);
        at->end = __shfl_sync(kFull, x.end, src);
    }
    return share;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 4608 bytes from global to shared memory; completion counts on `bar`
__device__ __forceinline__ void fetch_block(uint8_t *dst, const uint8_t *src, unsigned long long *bar)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(kQBlock) : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
                 "l"(src), "r"(kQBlock), "r"(smem_addr(bar))
                 : "memory");
}

// Wait for a phase of `bar`; gives up after a bounded number of tries.
__device__ __forceinline__ bool wait_block(unsigned long long *bar, uint32_t parity)
{
    for (int i = 0; i < (1 << 22); i++) {
        uint32_t ok;
        asm volatile(
            "{\n.reg .pred p;\n"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// d = c + a b: 16 x 16 times 16 x 8, halves in, fp32 sums
__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                         float c0, float c1, float c2, float c3)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// d = c + a b: 16 x 32 times 32 x 8, signed bytes in, 32-bit sums.  The sums
// start at kQaMagic, the bits of 1.5 2^23: read as fp32 they are 1.5 2^23 + the
// sum (below 2^22), so no conversion is needed.
constexpr uint32_t kQaMagic = 0x4b400000u;
__device__ __forceinline__ void imma16832(float2 d[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    uint32_t x, y, z, w;
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(kQaMagic));
    d[0] = make_float2(__uint_as_float(x), __uint_as_float(y));
    d[1] = make_float2(__uint_as_float(z), __uint_as_float(w));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// l 2^d where a factor 2^d may be below fp32's range.  References lie as far
// apart as the sizes of values (2^-80 for rows of zeros, see attend_blocks); a
// sum of values that drops out with the factor is too small to matter, the
// weights of such rows are not.
__device__ __forceinline__ float shifted(float l, float d)
{
    const float a = fmaxf(d, -100.0f);
    return l * ex2(a) * ex2(d - a);      // the second is 1 for most
}

__device__ __forceinline__ uint32_t pack_half2(float2 a)
{
    const __half2 h = __floats2half2_rn(a.x, a.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 halves(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2 *>(&a)); }
__device__ __forceinline__ float bf16_lo(uint32_t a) { return __uint_as_float(a << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t a) { return __uint_as_float(a & 0xffff0000u); }

// Two codes (nibble 0, or 1, of the bytes 0 and 2) as halves (c - 8) 2^-9: the
// bits c are the subnormal half c 2^-24, the upper nibble's 16 c 2^-24; one
// exact multiply-add makes either normal.
constexpr float kQaUnit = 512.0f;
__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return fma_half2(w & 0x000f000fu, 0x78007800u, 0xa400a400u); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return fma_half2(w & 0x00f000f0u, 0x68006800u, 0xa400a400u); }

// The reference maximum may lag the true one by 2^kQaLag, and weights are
// lifted by 2^kQaLift: at most 2^14, a half's range.  What a pair of halves
// drops of a weight is then at most 2^-37 of the largest one, 2^-17 over a
// million keys whose errors all point one way; each step of lag would double
// that, and raising the reference takes 2% of the time without any.
constexpr float kQaLag = 1.0f;
constexpr float kQaLift = 13.0f;

// q of one head as fixed point, in four signed bytes, of each group's largest
// magnitude: off by at most 2^-30 of that, and exact for a bf16 that is not below
// its 2^-22th part.  (One unit for all 128 channels would lose small ones beside a
// large one that the keys do not have, three bytes those of the same group: with
// one channel 1024 times the others the outputs were off by 3e-4.)  By one warp:
// lane l has channels 4l .. 4l + 3, 8 lanes a group.
__device__ __forceinline__ void stage_q(const float v[4], float scale2, uint32_t (*q)[4][8], float4 *qscale, int lane)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    // q 2^(156 - e) is below 2^30; a product is 16 (code - 8) times a digit of weight 2^24.  A query with an infinity
    // or NaN has NaN logits
    const uint32_t e = min(max(top >> 23, 30u), 254u);
    const float up = __uint_as_float((283u - e) << 23);
    if ((lane & 7) == 0)
        reinterpret_cast<float *>(qscale)[lane >> 3] = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : scale2 * __uint_as_float((e - 9u) << 23);
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; i++)          // bytes 3, 2, 1, 0: digits 0, 1, 2, 3
        d[i] = ((uint32_t)__float2int_rn(v[i] * up) + 0x00808080u) ^ 0x00808080u;
    const int r = lane >> 3, t = (lane & 7) >> 1;
#pragma unroll
    for (int k = 0; k < 4; k++)
#pragma unroll
        for (int h = 0; h < 2; h++)
            reinterpret_cast<uint16_t *>(&q[k][r][2 * t + h])[lane & 1] =
                (uint16_t)__byte_perm(d[h], d[h + 2], (uint32_t)(3 - k) | (uint32_t)(7 - k) << 4);
}

__device__ __forceinline__ void load_q(float v[4], const QuantAttendArgs &a, int p, int head, int lane)
{
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = ld_as_f32(a.q, ((int64_t)p * a.G + head) * kD + 4 * lane + i, a.is_bf16);
}

// Attention over a worker's blocks.
//
// A warp takes whole blocks of 32 keys from its own ring of bulk copies.
// A mask and a multiply-add make matrix operands of two codes.  (The masked
// bits are subnormal halves and would do as they are, but products of
// subnormals are summed with their leading zeros: errors of 2^-16.)
//   logits  S^T[16 x 8] = q[16 x 32] K^T[32 x 8] of bytes: rows are digits of
//           the heads' q, columns keys, one product per group of channels,
//           whose digits are joined and scaled by the group's scale.  Bytes
//           take 3 instructions for 8 codes (halves 9) and half the products,
//           and the sums are exact.
//   values  O^T[16 x 8] += V^T[16 x 16] w[16 x 8]: rows are channels, columns
//           heads, w = p times the value scale of the rows' group.
// A logit tile's fragment (head, two keys) is a value tile's weight fragment.
// A weight is a pair of halves (22 bits; one would cost 2^-12): up to 4 heads
// the low parts are the columns 4..7, else they are a second product.
// The reference maximum is of logit + exponent of the key's largest value
// scale, so that w, not p, is what stays within a half's range.
template <bool WIDE, int SPAN, int TURNS>
__device__ __forceinline__ void attend_blocks(const QuantAttendArgs &a, QaSmem &sm, const Place &at, uint32_t share)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, G = a.G;
    const int group = warp / SPAN, mate = warp % SPAN;           // worker within the CTA, warp within the worker
    const uint32_t worker = blockIdx.x * (kQaWarps / SPAN) + group;
    auto sync = [&]() {
        if (SPAN == kQaWarps) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * SPAN) : "memory");
    };
    const uint32_t x0 = at.start, end = at.end;
    if (end == 0) return;
    if (mate == 0 && lane == 0) sm.share[group] = share;
    int p = (int)at.pair;
    uint32_t first = at.first;           // first block of pair p
    const int64_t pair_blocks = a.c.n_cap / kQKeys;

    // the warp's blocks are x = mate (mod SPAN); copies run ahead of x
    uint32_t x = x0 + (mate + SPAN - x0 % SPAN) % SPAN;
    uint32_t fx = x, ffirst = first, fnb = block_count(a.c, p);
    int fp = p;
    auto fetch = [&](int s) {
        if (fx >= end) return;
        while (fx - ffirst >= fnb) {
            ffirst += fnb;
            fnb = block_count(a.c, ++fp);
        }
        if (lane == 0) fetch_block(sm.ring[warp][s], a.c.blocks + (fp * pair_blocks + (fx - ffirst)) * kQBlock, &sm.bar[warp][s]);
        fx += SPAN;
    };
    int slot = 0;
    uint32_t parity = 0;
    const int head = WIDE ? g : (g & 3);
    const float low = !WIDE && g >= 4 ? -1.0f : 0.0f;   // this column holds the weights' low parts

    // high_digit d[0] + low_digit d[1] without the sums' 1.5 2^23.  Sums are multiples of 16 below 2^20, so WIDE's are exact
    // and are joined with one rounding; else this is the rounding
    const float high_digit = WIDE || g < 4 ? 1.0f : 0x1p-8f, low_digit = WIDE ? 0x1p-8f : high_digit * 0x1p-16f;
    const float start = -12582912.0f * (high_digit + low_digit);
    auto joined = [&](const float2 d[2]) {
        return fma2(d[1], make_float2(low_digit, low_digit), fma2(d[0], make_float2(high_digit, high_digit), make_float2(start, start)));
    };

    constexpr int kHeads = (kMaxGroup + SPAN - 1) / SPAN;        // heads whose q a warp stages
    float qv[kHeads][4];
    auto q_of = [&](int turn, int h) { return (group * TURNS + (TURNS > 1 ? turn : 0)) * (WIDE ? kMaxGroup : 4) + h; };
    auto bring_q = [&](int pair) {
#pragma unroll
        for (int i = 0; i < kHeads; i++)
            if (mate + i * SPAN < G) load_q(qv[i], a, pair, mate + i * SPAN, lane);
    };
    auto put_q = [&](int turn) {
#pragma unroll
        for (int i = 0; i < kHeads; i++) {
            const int h = mate + i * SPAN;
            if (h < G) stage_q(qv[i], a.scale2, sm.q[q_of(turn, h)], &sm.qscale[group][turn][h], lane);
        }
    };
    bring_q(p);                          // ahead of the copies, which fill the memory's queues
#pragma unroll 1
    for (int s = 0; s < kQaStages; s++) fetch(s);
    put_q(0);
    sync();
    int turn = 0;
    while (first < end) {                // segments: pairs that have keys
        const int n = quant_len(a.c, p);
        const uint32_t nb = (uint32_t)(n + kQKeys - 1) / kQKeys, stop = min(end, first + nb);
        const bool has = x < stop;
        if (first >= x0 && mate == 0 && lane == 0) { // this worker has the pair's first block: where its partial results are
            const uint32_t share = sm.share[group] & 0x7fffffffu;
            a.parts[p] = make_uint2(worker, sm.share[group] >> 31 ? (nb + share - 1) / share : (first + nb - 1) / share - worker + 1);
        }
        float2 o[4][4];                  // channels 32r + {0, 16, 8, 24} + g, heads 2t and 2t + 1
        float m = -INFINITY;
        float2 l2 = make_float2(0.0f, 0.0f);
        int free_slot = -1;
        if (has) {
            // a product's rows g and g + 8 hold q's digits 0 and 1, and 2 and 3 (WIDE), or g / 4 and g / 4 + 2
            uint32_t qd[4][WIDE ? 8 : 4];
            const float4 qscale = head < G ? sm.qscale[group][turn][head] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int k = 0; k < (WIDE ? 4 : 2); k++) {
                    const uint2 d = *reinterpret_cast<const uint2 *>(&sm.q[q_of(turn, head)][WIDE ? k : (g >> 2) + 2 * k][r][2 * t]);
                    qd[r][2 * (k & 2) + (k & 1)] = head < G ? d.x : 0u;
                    qd[r][2 * (k & 2) + (k & 1) + 2] = head < G ? d.y : 0u;
                }
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int h = 0; h < 4; h++) o[r][h] = make_float2(0.0f, 0.0f);

#pragma unroll 1
            for (; x < stop; x += SPAN) {
                uint8_t *blk = sm.ring[warp][slot];
                if (!wait_block(&sm.bar[warp][slot], parity) && lane == 0) quant_late(a.c.status, p);
                const int b = (int)(x - first), valid = min(kQKeys, n - b * kQKeys);
                {   // scales as fp32 (zero behind the length), two groups of two keys a lane
                    const int pair = lane >> 1, half = lane & 1;
                    uint2 k = make_uint2(0, 0), v = make_uint2(0, 0);
                    const uint32_t *sk = reinterpret_cast<const uint32_t *>(blk + kQOffKs) + 4 * pair + half;
                    const uint32_t *sv = reinterpret_cast<const uint32_t *>(blk + kQOffVs) + 4 * pair + half;
                    if (2 * pair < valid) k.x = sk[0], v.x = sv[0];
                    if (2 * pair + 1 < valid) k.y = sk[2], v.y = sv[2];
                    sm.ks[warp][lane] = make_float4(bf16_lo(k.x), bf16_lo(k.y), bf16_hi(k.x), bf16_hi(k.y));
                    sm.vs[warp][lane] = make_float4(bf16_lo(v.x), bf16_lo(v.y), bf16_hi(v.x), bf16_hi(v.y));
                    // exponents, 0 for those of infinities and NaN
                    uint32_t ex = (v.x >> 7) & 0x00ff00ffu, ey = (v.y >> 7) & 0x00ff00ffu;
                    ex &= ~((((ex + 0x00010001u) >> 8) & 0x00010001u) * 255u);
                    ey &= ~((((ey + 0x00010001u) >> 8) & 0x00010001u) * 255u);
                    uint32_t e = __vmaxu2(__byte_perm(ex, ey, 0x5410), __byte_perm(ex, ey, 0x7632));   // (key, key + 1)
                    e = __vmaxu2(e, __shfl_xor_sync(kFull, e, 1));
                    sm.size[warp][lane] = fmaxf((float)((int)((e >> (16 * half)) & 0xffffu) - 126), -80.0f);
                    __syncwarp();
                }
                float2 z[4];             // keys 8i + 2t, + 1
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint4 kc = *reinterpret_cast<const uint4 *>(blk + (8 * i + g) * kQRow + 16 * t);
                    const float4 s01 = sm.ks[warp][2 * (4 * i + t)], s23 = sm.ks[warp][2 * (4 * i + t) + 1];
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        const uint32_t w = r == 0 ? kc.x : r == 1 ? kc.y : r == 2 ? kc.z : kc.w;
                        const uint32_t b0 = ((w << 4) & 0xf0f0f0f0u) ^ 0x80808080u, b1 = (w & 0xf0f0f0f0u) ^ 0x80808080u;   // 16 (code - 8)
                        float2 d[2], x;
                        imma16832(d, qd[r][0], qd[r][1], qd[r][2], qd[r][3], b0, b1);
                        x = joined(d);
                        if (WIDE) {
                            imma16832(d, qd[r][4], qd[r][5], qd[r][6], qd[r][7], b0, b1);
                            x = fma2(joined(d), make_float2(0x1p-16f, 0x1p-16f), x);
                        }
                        const float2 sc = r == 0 ? make_float2(s01.x, s01.y) : r == 1 ? make_float2(s01.z, s01.w)
                                        : r == 2 ? make_float2(s23.x, s23.y) : make_float2(s23.z, s23.w);
                        const float f = r == 0 ? qscale.x : r == 1 ? qscale.y : r == 2 ? qscale.z : qscale.w;
                        const float2 unit = mul2(sc, make_float2(f, f));
                        z[i] = r ? fma2(x, unit, z[i]) : mul2(x, unit);
                    }
                    if (!WIDE) z[i] = add2(z[i], make_float2(__shfl_xor_sync(kFull, z[i].x, 16), __shfl_xor_sync(kFull, z[i].y, 16)));
                }
                if (a.logits && g < G) {
                    float *zo = a.logits + ((p * pair_blocks + b) * G + g) * kQKeys + 2 * t;
#pragma unroll
                    for (int i = 0; i < 4; i++) *reinterpret_cast<float2 *>(zo + 8 * i) = z[i];
                }
                if (valid < kQKeys) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (8 * i + 2 * t >= valid) z[i].x = -INFINITY;
                        if (8 * i + 2 * t + 1 >= valid) z[i].y = -INFINITY;
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 e = add2(z[i], *reinterpret_cast<const float2 *>(&sm.size[warp][8 * i + 2 * t]));
                    top = fmaxf(top, fmaxf(e.x, e.y));
                }
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                if (__any_sync(kFull, top > m + kQaLag)) {     // rare: raise the reference maximum
                    const float to = top > m + kQaLag ? top : m;
                    const float d = to == -INFINITY ? 0.0f : m - to, f = ex2(d);
                    m = to;
                    l2 = make_float2(shifted(l2.x, d), shifted(l2.y, d));
                    const float2 fc = make_float2(__shfl_sync(kFull, f, 8 * t), __shfl_sync(kFull, f, 8 * t + 4));
#pragma unroll
                    for (int r = 0; r < 4; r++)
#pragma unroll
                        for (int h = 0; h < 4; h++) o[r][h] = mul2(o[r][h], fc);
                }
                const float off = m == -INFINITY ? 0.0f : kQaLift - m;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    z[i] = add2(z[i], make_float2(off, off));
                    z[i] = make_float2(ex2(z[i].x), ex2(z[i].y));
                    l2 = add2(l2, z[i]);
                }
                uint2 vc[2][4];          // codes of the keys 16u + 2t, + 1, + 8, + 9
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int key = 16 * u + 8 * (k >> 1) + 2 * t + (k & 1);
                        vc[u][k] = *reinterpret_cast<const uint2 *>(blk + kQOffV + key * kQRow + 8 * (g ^ v_turn(key)));
                    }
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    float d[2][4];
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        uint32_t bw[2], bl[2];
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            const float2 sc = reinterpret_cast<const float2 *>(&sm.vs[warp][2 * (8 * u + 4 * k + t)])[r];
                            const float2 w = mul2(z[2 * u + k], sc);
                            const uint32_t hi = pack_half2(w);
                            if (WIDE) {
                                bw[k] = hi;
                                bl[k] = pack_half2(fma2(halves(hi), make_float2(-1.0f, -1.0f), w));
                            } else {
                                bw[k] = pack_half2(fma2(halves(hi), make_float2(low, low), w));
                            }
                        }
                        // codes of the group's channels: halves (key 2t, key 2t + 1), and the keys 8 further
                        const uint32_t sel = (r & 1) ? 0x7632u : 0x5410u;
                        const uint32_t v0 = __byte_perm(r < 2 ? vc[u][0].x : vc[u][0].y, r < 2 ? vc[u][1].x : vc[u][1].y, sel);
                        const uint32_t v1 = __byte_perm(r < 2 ? vc[u][2].x : vc[u][2].y, r < 2 ? vc[u][3].x : vc[u][3].y, sel);
                        const uint32_t a0 = codes_lo(v0), a1 = codes_lo(v0 >> 8), a2 = codes_lo(v1), a3 = codes_lo(v1 >> 8);
                        const uint32_t c0 = codes_hi(v0), c1 = codes_hi(v0 >> 8), c2 = codes_hi(v1), c3 = codes_hi(v1 >> 8);
                        // matrix instructions cut their sums: a block's only, which are then added with rounding
                        mma16816(d[0], a0, a1, a2, a3, bw[0], bw[1], u ? d[0][0] : 0.0f, u ? d[0][1] : 0.0f, u ? d[0][2] : 0.0f, u ? d[0][3] : 0.0f);
                        mma16816(d[1], c0, c1, c2, c3, bw[0], bw[1], u ? d[1][0] : 0.0f, u ? d[1][1] : 0.0f, u ? d[1][2] : 0.0f, u ? d[1][3] : 0.0f);
                        if (WIDE) {
                            mma16816(d[0], a0, a1, a2, a3, bl[0], bl[1], d[0][0], d[0][1], d[0][2], d[0][3]);
                            mma16816(d[1], c0, c1, c2, c3, bl[0], bl[1], d[1][0], d[1][1], d[1][2], d[1][3]);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        o[r][2 * h] = add2(o[r][2 * h], make_float2(d[h][0], d[h][1]));
                        o[r][2 * h + 1] = add2(o[r][2 * h + 1], make_float2(d[h][2], d[h][3]));
                    }
                }
                __syncwarp();
                if (x + SPAN < stop) fetch(slot);
                else free_slot = slot;   // its block holds the warp's sums until they are merged
                if (++slot == kQaStages) {
                    slot = 0;
                    parity ^= 1u;
                }
            }
            // sums into the block consumed last: [column][channel]
            float *so = reinterpret_cast<float *>(sm.ring[warp][free_slot]);
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    const int c = 32 * r + 16 * (h & 1) + 8 * (h >> 1) + g;
                    so[2 * t * kQaCol + c] = o[r][h].x * kQaUnit;
                    so[(2 * t + 1) * kQaCol + c] = o[r][h].y * kQaUnit;
                }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            float l = l2.x + l2.y;
            l += __shfl_xor_sync(kFull, l, 1);
            l += __shfl_xor_sync(kFull, l, 2);
            if (t == 0) {
                sm.m[warp][g] = m;
                sm.l[warp][g] = l;
            }
        }
        if (lane == 0) sm.has[warp] = has ? free_slot : -1;
        int next = p + 1;                // the next segment's pair, and its q
        if (stop < end) {
            while (block_count(a.c, next) == 0) next++;
            bring_q(next);
        }
        sync();
        float *part = a.part + (int64_t)(p + worker) * G * kQPart;
#pragma unroll
        for (int h = mate; h < G; h += SPAN) {       // lane w < SPAN has warp w's reference and sum
            const int w = group * SPAN + lane % SPAN;
            const bool in = lane < SPAN && sm.has[w] >= 0;
            const float mw = in ? sm.m[w][h] : -INFINITY;
            float top = mw;
#pragma unroll
            for (int i = SPAN / 2; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
            const float d = mw - (top == -INFINITY ? 0.0f : top), f = in ? ex2(d) : 0.0f;
            float l = in ? shifted(sm.l[w][h], d) : 0.0f;
#pragma unroll
            for (int i = SPAN / 2; i; i >>= 1) l += __shfl_xor_sync(kFull, l, i);
            if (lane < SPAN) sm.factor[w][h] = f;
            if (lane == 0) {
                part[h * kQPart + kD] = top - kQaLift;
                part[h * kQPart + kD + 1] = l;
            }
        }
        sync();
        for (int e = 32 * mate + lane; e < G * kD; e += 32 * SPAN) {
            const int h = e / kD, c = e % kD;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < SPAN; i++) {
                const int w = group * SPAN + i;
                if (sm.has[w] >= 0) {
                    const float *so = reinterpret_cast<const float *>(sm.ring[w][sm.has[w]]);
                    sum = fmaf(sm.factor[w][h], WIDE ? so[h * kQaCol + c] : so[h * kQaCol + c] + so[(h + 4) * kQaCol + c], sum);
                }
            }
            part[h * kQPart + c] = sum;
        }
        turn ^= 1;
        if (stop < end) put_q(turn);
        sync();
        if (free_slot >= 0) fetch(free_slot);
        first += nb;
        p = next;
    }
}

// A worker is a CTA, or 4 warps of one.  Large workers leave fewer partial
// results; small ones lose less to rounds that do not fill their warps, and
// there are enough of them to take one pair each where lengths differ much.
// kFewPairs: large by pairs, else large evenly.  kSomePairs: large by pairs, else
// small by pairs, else large evenly (96 ragged pairs of up to 9001 keys: 29 us,
// 51 without the small; their code costs a long pair's loop registers: 64 pairs
// of 131072 keys 265 us for 263, 8 of 1048576 314 for 303, hence not for few
// pairs).  kManyPairs: small by pairs, else small evenly (256 pairs of 577 keys:
// 17 us, 20 large).
enum Workers { kFewPairs, kSomePairs, kManyPairs };
constexpr int kQaFewPairs = 32, kQaManyPairs = 129;      // up to, and from
template <bool WIDE, Workers KIND>
__global__ void __launch_bounds__(kQaThreads, 1) k_quant_attend(QuantAttendArgs a)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    QaSmem &sm = *reinterpret_cast<QaSmem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (lane < kQaStages) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&sm.bar[warp][lane])) : "memory");
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");     // the barriers, and rows that earlier kernels wrote
    pdl_trigger();

    // the worker's blocks, and the pair of the first
    Place at;
    uint32_t share = 0;
    const int ctas = (int)gridDim.x;
    bool large = KIND != kManyPairs;
    if (large) share = plan_pairs<KIND == kFewPairs ? 1 : 4, kQaWarps>(a.c, ctas, blockIdx.x, warp, lane, sm.fits[0], &at);
    if (KIND != kFewPairs && share == 0) {
        const uint32_t worker = blockIdx.x * kQaGroups + warp / kQaFew;
        share = plan_pairs<8, kQaFew>(a.c, ctas * kQaGroups, worker, warp, lane, sm.fits[1], &at);
        if (share > 0) large = false;
    }
    if (share > 0) {
        share |= 0x80000000u;
    } else {
        const int groups = large ? 1 : kQaGroups;
        const uint32_t total = count_blocks(a.c, sm.ws), worker0 = blockIdx.x * groups;
        share = even_share(total, ctas * groups, kQaWarps / groups);
        if (worker0 * share >= total) return;
        if (tid < groups) sm.place[tid].end = 0;         // no work unless there are blocks for it
        for (uint32_t base = 0, c = 0;; c += kQaThreads) {
            const uint32_t v = c + tid < (uint32_t)a.c.bh ? block_count(a.c, c + tid) : 0u;
            uint32_t sum, last = 0;
            const uint32_t before = base + block_excl_scan<kQaThreads>(v, sm.ws, &sum);
            for (int j = 0; j < groups; j++) {
                const uint32_t x = (worker0 + j) * share;
                if (x >= before && x - before < v) sm.place[j] = Place{c + tid, before, x, min(total, x + share)};
                if (x < total) last = x;
            }
            base += sum;
            if (base > last) break;
        }
        __syncthreads();
        at = sm.place[large ? 0 : warp / kQaFew];
    }
    if (KIND == kManyPairs) attend_blocks<WIDE, kQaFew, 2>(a, sm, at, share);
    else if (KIND == kFewPairs || large) attend_blocks<WIDE, kQaWarps, 2>(a, sm, at, share);
    else attend_blocks<WIDE, kQaFew, 1>(a, sm, at, share);       // one pair: no q of a next one
}

// Joined partial results of a head: reference, weights' sum, one channel's sum.
struct Joined {
    float top, l, o;
    __device__ float ref() const { return top == -INFINITY ? 0.0f : top; }
    __device__ float out() const { return l == 0.0f ? 0.0f : o / l; }
    __device__ float lse() const { return (log2f(l) + ref()) * 0.69314718055994531f; }
};

// Of the head's ns partial results at pg those first, first + step ..: N at a
// time, all that is needed of them in flight at once.  Every thread sums the
// head's weights too, one round trip to memory instead of two and a barrier (64
// ragged pairs: 33 us for 35).  More than 6 at a time cost more instructions
// than they save in latency (8 pairs of 18 partial results: 24.2 us, 24.7 by 8,
// 25.8 by 18; 256 pairs of 2: 20.0 us, 22.5 by 8).
template <int N>
__device__ __forceinline__ Joined join_parts(const float *pg, int64_t stride, int ns, int c, int first = 0, int step = 1)
{
    Joined j = {-INFINITY, 0.0f, 0.0f};
    for (int s = first; s < ns; s += N * step) {
        float m[N], w[N], x[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float *q = pg + (s + i * step) * stride;
            const bool in = s + i * step < ns;
            m[i] = in ? q[kD] : -INFINITY;
            w[i] = in ? q[kD + 1] : 0.0f;
            x[i] = in ? q[c] : 0.0f;
        }
        const float old = j.top;
#pragma unroll
        for (int i = 0; i < N; i++) j.top = fmaxf(j.top, m[i]);
        const float ref = j.ref();
        j.l = shifted(j.l, old - ref);
        j.o *= ex2(old - ref);
#pragma unroll
        for (int i = 0; i < N; i++) {
            j.l += shifted(w[i], m[i] - ref);
            j.o = fmaf(ex2(m[i] - ref), x[i], j.o);
        }
    }
    return j;
}

// Merge of a pair's partial results (the first a.outs CTAs) and its part of acc
// (the others, kQmKeys keys each).  The lengths are read before the attention
// kernel has ended: it waited for whatever wrote them.
template <bool WIDE>
__global__ void __launch_bounds__(kQmThreads, WIDE ? 3 : 4) k_quant_merge(QuantAttendArgs a)
{
    constexpr int kHeads = WIDE ? kMaxGroup : 4;
    __shared__ float s_lse[kHeads];
    const int tid = threadIdx.x, p = blockIdx.y, G = a.G;
    const int n = quant_len(a.c, p);
    const int outs = a.outs;
    const bool is_out = (int)blockIdx.x < outs;
    const int64_t k0 = (int64_t)((int)blockIdx.x - outs) * kQmKeys;
    if (!is_out && k0 >= n) return;
    pdl_wait();
    if (blockIdx.x == 0 && tid == 0 && quant_len_bad(a.c, p)) quant_devchk(a.c.status, p);
    if (n == 0) {
        for (int e = (int)blockIdx.x * kQmThreads + tid; e < G * kD; e += outs * kQmThreads) a.out[(int64_t)p * G * kD + e] = 0.0f;
        if (blockIdx.x == 0 && tid < G && a.lse) a.lse[(int64_t)p * G + tid] = -INFINITY;
        return;
    }
    const uint2 *parts = a.parts + p;    // slots p + x .. p + x + y - 1 have the pair's partial results
    const int warp = tid >> 5, lane = tid & 31;
    const int64_t stride = (int64_t)G * kQPart;
    if (is_out) {
        const uint2 at = *parts;
        const int ns = (int)at.y;
        if (a.sliced) {                  // 32 channels of a head a CTA, each warp a share of the partial results
            constexpr int kSlices = kQmThreads / 32, kParts = kD / 32;
            __shared__ Joined s_join[kSlices][32];
            const int h = (int)blockIdx.x / kParts, c = (int)blockIdx.x % kParts * 32 + lane;
            const float *pg = a.part + (int64_t)(p + at.x) * stride + h * kQPart;
            s_join[warp][lane] = ns <= 2 * kSlices ? join_parts<2>(pg, stride, ns, c, warp, kSlices) : join_parts<4>(pg, stride, ns, c, warp, kSlices);
            __syncthreads();
            if (warp > 0) return;
            Joined j = {-INFINITY, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kSlices; w++) j.top = fmaxf(j.top, s_join[w][lane].top);
#pragma unroll
            for (int w = 0; w < kSlices; w++) {
                const float d = s_join[w][lane].top - j.ref();
                j.l += shifted(s_join[w][lane].l, d);
                j.o = fmaf(ex2(d), s_join[w][lane].o, j.o);
            }
            a.out[((int64_t)p * G + h) * kD + c] = j.out();
            if (c == 0 && a.lse) a.lse[(int64_t)p * G + h] = j.lse();
            return;
        }
        for (int e = (int)blockIdx.x * kQmThreads + tid; e < G * kD; e += outs * kQmThreads) {
            const float *pg = a.part + (int64_t)(p + at.x) * stride + e / kD * kQPart;
            const Joined j = ns <= 2 ? join_parts<2>(pg, stride, ns, e % kD) : join_parts<6>(pg, stride, ns, e % kD);
            a.out[(int64_t)p * G * kD + e] = j.out();
            if (e % kD == 0 && a.lse) a.lse[(int64_t)p * G + e / kD] = j.lse();
        }
        return;
    }
    // 4 keys a thread: all heads' logits and the sums in flight at once, the first ones beside the log-sums'
    float *acc = a.c.acc + (int64_t)p * a.c.n_cap;
    const bool vec = (uintptr_t)acc % 16 == 0;
    const int64_t end = min((int64_t)n, k0 + kQmKeys);
    auto load = [&](int64_t k, float4 x[kHeads], float4 *sum) {
        const float *z = a.logits + ((int64_t)p * (a.c.n_cap / kQKeys) + k / kQKeys) * G * kQKeys + k % kQKeys;
#pragma unroll
        for (int g = 0; g < kHeads; g++)
            if (g < G) x[g] = __ldcs(reinterpret_cast<const float4 *>(z + g * kQKeys));
        if (vec && k + 4 <= n) *sum = *reinterpret_cast<const float4 *>(acc + k);
    };
    auto add = [&](int64_t k, const float4 x[kHeads], const float4 &sum) {
        float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int g = 0; g < kHeads; g++)
            if (g < G) {
                const float lse = s_lse[g];
                w.x += ex2(x[g].x - lse);
                w.y += ex2(x[g].y - lse);
                w.z += ex2(x[g].z - lse);
                w.w += ex2(x[g].w - lse);
            }
        if (vec && k + 4 <= n) {
            *reinterpret_cast<float4 *>(acc + k) = make_float4(sum.x + w.x, sum.y + w.y, sum.z + w.z, sum.w + w.w);
        } else {
            acc[k] += w.x;
            if (k + 1 < n) acc[k + 1] += w.y;
            if (k + 2 < n) acc[k + 2] += w.z;
            if (k + 3 < n) acc[k + 3] += w.w;
        }
    };
    float4 x[kHeads], sum;
    int64_t k = k0 + 4 * tid;
    if (k < end) load(k, x, &sum);
    if (warp < G) {                      // head `warp`: its log-sum
        const uint2 at = *parts;
        const int ns = (int)at.y;
        const float *pg = a.part + (int64_t)(p + at.x) * stride + warp * kQPart + kD;
        float m = -INFINITY;
        for (int s = lane; s < ns; s += 32) m = fmaxf(m, pg[s * stride]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        const float ref = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
        for (int s = lane; s < ns; s += 32) l += shifted(pg[s * stride + 1], pg[s * stride] - ref);
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
        if (lane == 0) s_lse[warp] = l == 0.0f ? INFINITY : log2f(l) + ref;
    }
    static_assert(kQmThreads / 32 >= kHeads, "a warp for each head");
    __syncthreads();
    while (k < end) {
        add(k, x, sum);
        k += 4 * kQmThreads;
        if (k < end) load(k, x, &sum);
    }
}

cudaError_t launch_quant_attend(const QuantAttendArgs &args, int num_sms, cudaStream_t s)
{
    static std::atomic<int> done[6][kMaxDevices];
    QuantAttendArgs a = args;
    const bool wide = a.G > 4;
    const Workers kind = a.c.bh <= kQaFewPairs ? kFewPairs : a.c.bh < kQaManyPairs ? kSomePairs : kManyPairs;
    auto kern = kind == kFewPairs    ? (wide ? k_quant_attend<true, kFewPairs> : k_quant_attend<false, kFewPairs>)
                : kind == kSomePairs ? (wide ? k_quant_attend<true, kSomePairs> : k_quant_attend<false, kSomePairs>)
                                     : (wide ? k_quant_attend<true, kManyPairs> : k_quant_attend<false, kManyPairs>);
    const int ctas = min(num_sms, kQMaxWorkers / kQaGroups);
    // q of two pairs for one worker or 4, or of one for 4; no more, the rest is cache (32 KB more: 8 pairs of 32768 keys
    // 24 us for 22)
    const int staged = (kind == kFewPairs ? 2 : kind == kSomePairs ? 4 : 8) * (wide ? kMaxGroup : 4);
    const size_t smem = offsetof(QaSmem, q) + staged * sizeof(QaSmem::q) / (kQaGroups * 2 * kMaxGroup);
    cudaError_t e = dyn_smem_limit(kern, (int)smem, done[2 * kind + wide]);
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(kQaThreads), smem, s, a);
    if (e != cudaSuccess) return e;
    const unsigned parts = a.accumulate ? (unsigned)((a.c.n_cap + kQmKeys - 1) / kQmKeys) : 0u;
    // few pairs have many partial results each: 32 channels of a head a CTA, if the CTAs are all there at once (1 pair of
    // 131072 keys: 17 us for 27; 16 of 4096: 10.0 for 11.9; 2 of 500 8.9 for 8.5); others have fewer: one pass a CTA; many
    // have few: fewer CTAs (256 pairs: 22 us for 24)
    a.sliced = a.c.n_cap >= 8 * min_share(kQaWarps) * kQKeys && a.c.bh * a.G <= num_sms &&
               a.c.bh * (a.G * (kD / 32) + (int64_t)parts) <= 4 * num_sms;
    a.outs = a.sliced ? a.G * (kD / 32) : a.c.bh < num_sms ? (a.G + kQmHeads - 1) / kQmHeads : 1;
    return launch_pdl(a.G > 4 ? k_quant_merge<true> : k_quant_merge<false>, dim3(a.outs + parts, a.c.bh), dim3(kQmThreads), 0, s, a);
}

}  // namespace pk
