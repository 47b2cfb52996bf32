// pk_quant.cuh -- the 4-bit KV cache: block layout, device helpers and kernel
// argument blocks.  Not part of the public C-ABI.
#pragma once

#include "pk_internal.cuh"

namespace pk {

constexpr int kQKeys = PK_QUANT_KEYS;              // keys per block (32)
constexpr int kQBlock = PK_QUANT_BLOCK_BYTES;      // bytes per block (4608)
constexpr int kQRow = kD / 2;                      // code bytes of a row (64)
constexpr int kQGroups = 4;                        // groups of 32 channels, one scale each
constexpr int kQOffV = kQKeys * kQRow;             // V codes
constexpr int kQOffKs = 2 * kQKeys * kQRow;        // K scales
constexpr int kQOffVs = kQOffKs + kQKeys * kQGroups * 2;   // V scales
static_assert(kQOffVs + kQKeys * kQGroups * 2 == kQBlock, "block layout is part of the documented contract");

// V rows: 8-byte chunk c of key j is held at chunk place c ^ v_turn(j)
__host__ __device__ __forceinline__ int v_turn(int j) { return (j & 2) << 1; }

struct QuantCache {
    uint8_t *blocks;
    int32_t *lens;
    float *acc;
    int32_t *status;
    int64_t n_cap;
    int32_t bh;
};

// Record a device-check failure of pair p (first writer wins) without trapping.
__device__ __forceinline__ void quant_devchk(int32_t *status, int p)
{
    if (status && atomicCAS(status, 0, (int)PK_ERR_DEVICE_CHECK) == 0) status[1] = p;
}
// ... or that a bounded wait for one of its copies gave up.
__device__ __forceinline__ void quant_late(int32_t *status, int p)
{
    if (status && atomicCAS(status, 0, (int)PK_ERR_TIMEOUT) == 0) status[1] = p;
}

// Length of pair p within [0, n_cap].
__device__ __forceinline__ int quant_len(const QuantCache &c, int p)
{
    const int n = c.lens[p];
    return n < 0 ? 0 : (int64_t)n > c.n_cap ? (int)c.n_cap : n;
}
__device__ __forceinline__ bool quant_len_bad(const QuantCache &c, int p)
{
    const int n = c.lens[p];
    return n < 0 || (int64_t)n > c.n_cap;
}

__device__ __forceinline__ float bf16_bits_f32(uint32_t b) { return __uint_as_float(b << 16); }

struct QuantRowsArgs {
    QuantCache c;
    const void *k, *v;       // append: rows in; read back: rows out (cast)
    int64_t n_rows, stride;  // rows taken / rows between pairs
    const int32_t *at;       // first slot per pair, or null
    int32_t own_at;          // append: `at` does not overlap the lengths
    int32_t is_bf16;
    int32_t vec;             // bytes on whose boundary the rows lie: 32, 16 or 0 (less)
};

// Attention splits the pairs' blocks, laid end to end, over the CTAs
// ("workers") whatever the lengths.  A pair's segment in a worker leaves one
// partial result in slot pair + worker: consecutive segments differ in at
// least one of the two, so slots are never shared.
constexpr int kQMaxWorkers = 1024;
constexpr int kQPart = kD + 2;           // floats of a head's partial: sums, then reference maximum and weight sum

struct QuantAttendArgs {
    QuantCache c;
    const void *q;           // [bh][G][D]
    float *out;              // [bh][G][D]
    float *lse;              // [bh][G] or null
    float *part;             // [bh + kQMaxWorkers][G][kQPart]
    uint2 *parts;            // [bh]: first worker and number of partial results of a pair that has keys
    float *logits;           // [bh][n_cap / 32][G][32] (log2 units) when accumulating, else null
    int32_t G, is_bf16, accumulate;
    int32_t outs;            // merge kernel: CTAs per pair that write outputs
    int32_t sliced;          // ... of 32 channels of a head each
    float scale2;            // softmax scale * log2(e)
};

struct QuantEvictArgs {
    QuantCache src, dst;
    int64_t budget, sink, recent;
    int32_t *keep;           // [bh][budget] or null
};

cudaError_t launch_quant_append(const QuantRowsArgs &a, cudaStream_t s);
cudaError_t launch_quant_rows(const QuantRowsArgs &a, cudaStream_t s);
cudaError_t launch_quant_attend(const QuantAttendArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_quant_evict(const QuantEvictArgs &a, cudaStream_t s);

// two fp32 operations in one instruction
__device__ __forceinline__ unsigned long long as_u64(float2 a)
{
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 as_f2(unsigned long long a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_f2(r);
}

}  // namespace pk
