// k_quant_evict.cu -- eviction from the 4-bit KV cache by accumulated weight.
//
// Of a pair's keys the first `sink` and last `recent` stay; of the others the
// heaviest, by a radix select of the threshold weight over the ordered bits of
// acc, ties to lower slots.  One CTA per pair.
#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace pk {

constexpr int kQeThreads = 1024;

// ordered bits of a weight; NaN sorts below everything
__device__ __forceinline__ uint32_t weight_key(float x)
{
    return x != x ? 0u : ord_f32(x + 0.0f);
}

// one row of slot j from src to slot o of dst (pair bases), by one thread
__device__ __forceinline__ void copy_row(const uint8_t *src, int64_t j, uint8_t *dst, int64_t o)
{
    const uint8_t *b = src + j / kQKeys * kQBlock;
    uint8_t *d = dst + o / kQKeys * kQBlock;
    const int x = (int)(j % kQKeys), y = (int)(o % kQKeys);
#pragma unroll
    for (int c = 0; c < 4; c++)
        *reinterpret_cast<uint4 *>(d + y * kQRow + 16 * c) = *reinterpret_cast<const uint4 *>(b + x * kQRow + 16 * c);
#pragma unroll
    for (int c = 0; c < 8; c++)
        *reinterpret_cast<uint2 *>(d + kQOffV + y * kQRow + 8 * (c ^ v_turn(y))) =
            *reinterpret_cast<const uint2 *>(b + kQOffV + x * kQRow + 8 * (c ^ v_turn(x)));
    *reinterpret_cast<uint2 *>(d + kQOffKs + 8 * y) = *reinterpret_cast<const uint2 *>(b + kQOffKs + 8 * x);
    *reinterpret_cast<uint2 *>(d + kQOffVs + 8 * y) = *reinterpret_cast<const uint2 *>(b + kQOffVs + 8 * x);
}

__global__ void __launch_bounds__(kQeThreads) k_quant_evict(QuantEvictArgs a)
{
    __shared__ uint32_t s_hist[256];
    __shared__ uint32_t s_ws[kQeThreads / 32 + 1];
    __shared__ uint32_t s_digit, s_need;
    const int p = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    const int n = quant_len(a.src, p);
    if (tid == 0 && quant_len_bad(a.src, p)) quant_devchk(a.src.status, p);
    const float *acc = a.src.acc + (int64_t)p * a.src.n_cap;
    const bool all = n <= a.budget;
    const int lo = all ? n : (int)a.sink, hi = all ? n : n - (int)a.recent;   // contested slots
    uint32_t need = all ? 0u : (uint32_t)(a.budget - a.sink - a.recent);
    // threshold key T: the need-th largest; `need` ends as the ties to keep
    uint32_t prefix = 0, mask = 0;
    bool none = need == 0;
    if (!none) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kQeThreads) s_hist[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kQeThreads) {
                const uint32_t k = weight_key(acc[i]);
                if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                uint32_t left = need;
                int d = 255;
                for (; d > 0 && s_hist[d] < left; d--) left -= s_hist[d];
                s_digit = (uint32_t)d;
                s_need = left;
            }
            __syncthreads();
            prefix |= s_digit << shift;
            mask |= 255u << shift;
            need = s_need;
            __syncthreads();
        }
    }
    // kept slots in order
    const uint8_t *src = a.src.blocks + (int64_t)p * (a.src.n_cap / kQKeys) * kQBlock;
    uint8_t *dst = a.dst.blocks + (int64_t)p * (a.dst.n_cap / kQKeys) * kQBlock;
    uint32_t out = 0, ties = 0;
    for (int64_t c = 0; c < n; c += kQeThreads) {
        const int64_t i = c + tid;
        bool keep = false, tie = false;
        if (i < n) {
            if (i < lo || i >= hi) keep = true;
            else if (!none) {
                const uint32_t k = weight_key(acc[i]);
                keep = k > prefix;
                tie = k == prefix;
            }
        }
        uint32_t total;
        const uint32_t before = block_excl_scan<kQeThreads>(tie ? 1u : 0u, s_ws, &total);
        if (tie && ties + before < need) keep = true;
        ties += total;
        const uint32_t o = out + block_excl_scan<kQeThreads>(keep ? 1u : 0u, s_ws, &total);
        out += total;
        if (keep) {
            copy_row(src, i, dst, o);
            if (a.keep) a.keep[p * a.budget + o] = (int32_t)i;
            if (a.dst.acc) a.dst.acc[p * a.dst.n_cap + o] = acc[i];
        }
    }
    if (a.keep)
        for (int64_t o = out + tid; o < a.budget; o += kQeThreads) a.keep[p * a.budget + o] = -1;
    if (tid == 0) a.dst.lens[p] = (int32_t)out;
}

cudaError_t launch_quant_evict(const QuantEvictArgs &a, cudaStream_t s)
{
    return launch_pdl(k_quant_evict, dim3(a.src.bh), dim3(kQeThreads), 0, s, a);
}

}  // namespace pk
