// k_quant_rows.cu -- rows into and out of the 4-bit KV cache.
//
// Append: scale_r = bf16(max|x| / 7) over a group of 32 channels, code = 8 +
// round(x / scale) (ties to even, clamped to -7..7).  Reads 2 D es bytes per
// key and writes 144; read-back the other way round.  Both are bound by
// memory.
#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace pk {

constexpr int kQrThreads = 256;
constexpr int kQrRows = 64;              // rows (K and V) per CTA

// Code 0..15 of x for a group scale s > 0 with inv = 1 / s (both scaled out of
// the subnormal range by the caller).  rintf(x inv) can only be wrong next to
// a border (k + 1/2) s; r = x - k s is exact there (k s has 12 bits, and x is
// a multiple of a unit >= 2^-25 s once |x| >= s / 2), so comparing 2 |r| with
// s decides the border and its tie exactly.
__device__ __forceinline__ uint32_t quant_code(float x, float s, float inv)
{
    float k = rintf(x * inv);
    const float r = fmaf(-k, s, x), d = 2.0f * fabsf(r);
    if (d > s || (d == s && ((int)k & 1))) k += r > 0.0f ? 1.0f : -1.0f;
    return (uint32_t)(8 + (int)fminf(fmaxf(k, -7.0f), 7.0f));
}

// Scale of a group from its largest magnitude m (NaN if the group holds a
// NaN): bf16 bits; an infinity or NaN gives NaN.  Division and both roundings
// are the documented ones (fp32, then bf16, to nearest even).
__device__ __forceinline__ uint32_t quant_scale_bits(float m)
{
    if (!(m < INFINITY)) return 0x7fffu;
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(m, 7.0f)));
}

// largest magnitude that keeps a NaN (fmaxf would drop it)
__device__ __forceinline__ float max_mag(float a, float b)
{
    return (b != b || b > a) ? b : a;
}

__global__ void __launch_bounds__(kQrThreads) k_quant_append(QuantRowsArgs a)
{
    const int p = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int64_t at = a.at ? a.at[p] : a.c.lens[p];
    const bool fits = at >= 0 && at + a.n_rows <= a.c.n_cap;
    if (fits) {
        const int64_t r0 = (int64_t)blockIdx.x * kQrRows;
        uint8_t *pair = a.c.blocks + (int64_t)p * (a.c.n_cap / kQKeys) * kQBlock;
        // one warp per row; lane (r, g) = (lane / 8, lane % 8) of group r
        const int r = lane >> 3, g = lane & 7;
        for (int it = warp; it < 2 * kQrRows; it += kQrThreads / 32) {
            const int64_t i = r0 + (it >> 1);
            const bool is_v = it & 1;
            if (i >= a.n_rows) break;
            const int64_t slot = at + i;
            const int j = (int)(slot % kQKeys);
            uint8_t *blk = pair + slot / kQKeys * kQBlock;
            const void *src = is_v ? a.v : a.k;
            const int64_t base = ((int64_t)p * a.stride + i) * kD + 32 * r;
            // K: channels 4g .. 4g + 3 of the group; V: g, g + 8, g + 16, g + 24
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = ld_as_f32(src, base + (is_v ? g + 8 * e : 4 * g + e), a.is_bf16);
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; e++) m = max_mag(m, fabsf(x[e]));
#pragma unroll
            for (int h = 1; h <= 4; h <<= 1) m = max_mag(m, __shfl_xor_sync(kFull, m, h));
            const uint32_t sb = quant_scale_bits(m);
            float s = bf16_bits_f32(sb);
            uint32_t code = 0x8888u;
            if (s > 0.0f) {
                float up = 1.0f;
                if (s < 1e-18f) up = 18446744073709551616.0f;    // 2^64: 1 / s stays finite
                s *= up;
                const float inv = __fdiv_rn(1.0f, s);
                code = 0;
#pragma unroll
                for (int e = 0; e < 4; e++) code |= quant_code(x[e] * up, s, inv) << (4 * e);
            }
            if (is_v) {
                *reinterpret_cast<uint16_t *>(blk + kQOffV + j * kQRow + 8 * (g ^ v_turn(j)) + 2 * r) = (uint16_t)code;
                if (g == 0) *reinterpret_cast<uint16_t *>(blk + kQOffVs + 8 * j + 2 * r) = (uint16_t)sb;
            } else {
                *reinterpret_cast<uint16_t *>(blk + j * kQRow + 16 * (g >> 1) + 4 * r + 2 * (g & 1)) = (uint16_t)code;
                if (g == 0) *reinterpret_cast<uint16_t *>(blk + kQOffKs + 8 * j + 2 * r) = (uint16_t)sb;
            }
        }
        if (a.c.acc)
            for (int i = threadIdx.x; i < kQrRows && r0 + i < a.n_rows; i += kQrThreads)
                a.c.acc[(int64_t)p * a.c.n_cap + at + r0 + i] = 0.0f;
    }
    if (gridDim.x == 1) {                // every thread has read lens: the length may change
        __syncthreads();
        if (threadIdx.x == 0) {
            if (fits) a.c.lens[p] = (int32_t)(at + a.n_rows);
            else quant_devchk(a.c.status, p);
        }
    }
}

// New lengths after an append of several CTAs per pair.
__global__ void k_quant_lens(QuantRowsArgs a)
{
    pdl_wait();
    const int p = blockIdx.x * blockDim.x + threadIdx.x;
    if (p >= a.c.bh) return;
    const int64_t at = a.at ? a.at[p] : a.c.lens[p];
    if (at >= 0 && at + a.n_rows <= a.c.n_cap) a.c.lens[p] = (int32_t)(at + a.n_rows);
    else quant_devchk(a.c.status, p);
}

__global__ void __launch_bounds__(kQrThreads) k_quant_rows(QuantRowsArgs a)
{
    const int p = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int64_t at = a.at ? a.at[p] : 0;
    const int n = quant_len(a.c, p);
    if (blockIdx.x == 0 && threadIdx.x == 0 && quant_len_bad(a.c, p)) quant_devchk(a.c.status, p);
    const int64_t r0 = (int64_t)blockIdx.x * kQrRows;
    const uint8_t *pair = a.c.blocks + (int64_t)p * (a.c.n_cap / kQKeys) * kQBlock;
    const int r = lane >> 3, g = lane & 7;
    for (int it = warp; it < 2 * kQrRows; it += kQrThreads / 32) {
        const int64_t i = r0 + (it >> 1), slot = at + i;
        if (i >= a.n_rows) break;
        if (slot < 0 || slot >= n) continue;
        const bool is_v = it & 1;
        const int j = (int)(slot % kQKeys);
        const uint8_t *blk = pair + slot / kQKeys * kQBlock;
        const uint32_t code = *reinterpret_cast<const uint16_t *>(
            is_v ? blk + kQOffV + j * kQRow + 8 * (g ^ v_turn(j)) + 2 * r
                 : blk + j * kQRow + 16 * (g >> 1) + 4 * r + 2 * (g & 1));
        const float s = bf16_bits_f32(*reinterpret_cast<const uint16_t *>(blk + (is_v ? kQOffVs : kQOffKs) + 8 * j + 2 * r));
        void *dst = const_cast<void *>(is_v ? a.v : a.k);
        const int64_t base = ((int64_t)p * a.stride + i) * kD + 32 * r;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float x = (float)((int)((code >> (4 * e)) & 15u) - 8) * s;
            const int64_t o = base + (is_v ? g + 8 * e : 4 * g + e);
            if (a.is_bf16) reinterpret_cast<__nv_bfloat16 *>(dst)[o] = __float2bfloat16_rn(x);
            else reinterpret_cast<float *>(dst)[o] = x;
        }
    }
}

cudaError_t launch_quant_append(const QuantRowsArgs &a, cudaStream_t s)
{
    const unsigned tiles = (unsigned)((a.n_rows + kQrRows - 1) / kQrRows);
    cudaError_t e = launch_pdl(k_quant_append, dim3(tiles, a.c.bh), dim3(kQrThreads), 0, s, a);
    if (e == cudaSuccess && tiles > 1)
        e = launch_pdl(k_quant_lens, dim3((a.c.bh + 255) / 256), dim3(256), 0, s, a);
    return e;
}

cudaError_t launch_quant_rows(const QuantRowsArgs &a, cudaStream_t s)
{
    const unsigned tiles = (unsigned)((a.n_rows + kQrRows - 1) / kQrRows);
    return launch_pdl(k_quant_rows, dim3(tiles, a.c.bh), dim3(kQrThreads), 0, s, a);
}

}  // namespace pk
