// k_quant_rows.cu -- rows into and out of the 4-bit KV cache.
//
// Append: scale_r = bf16(max|x| / 7) over a group of 32 channels, code = 8 +
// round(x / scale) (ties to even, clamped to -7..7).  Reads 2 D es bytes per
// key and writes 144; read-back the other way round.  Both are bound by
// memory.
#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace pk {

constexpr int kQrWarps = 8;
constexpr int kQrThreads = 32 * kQrWarps;

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
    float q;
    if (m > 1e-30f) {
        // m / 7 to nearest by one step from the rounded reciprocal (Markstein 1990), exact for every normal m / 7
        constexpr float kSeventh = 1.0f / 7.0f;
        q = m * kSeventh;
        q = fmaf(fmaf(-7.0f, q, m), kSeventh, q);
    } else {
        q = __fdiv_rn(m, 7.0f);
    }
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(q));
}

// 8 consecutive elements i .. i + 7 of a bf16 or fp32 array, as they lie
struct Raw8 {
    uint32_t w[8];                       // fp32, or 4 words of 2 bf16
};
template <bool BF16>
__device__ __forceinline__ Raw8 load8(const void *p, int64_t i, int vec)
{
    Raw8 x;
    if (BF16) {
        const __nv_bfloat16 *b = reinterpret_cast<const __nv_bfloat16 *>(p) + i;
        if (vec) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(b));
            x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(b);
#pragma unroll
            for (int e = 0; e < 4; e++) x.w[e] = h[2 * e] | (uint32_t)h[2 * e + 1] << 16;
        }
    } else {
        const uint32_t *f = reinterpret_cast<const uint32_t *>(p) + i;
        if (vec) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(f)), v = __ldcs(reinterpret_cast<const uint4 *>(f) + 1);
            x.w[0] = u.x, x.w[1] = u.y, x.w[2] = u.z, x.w[3] = u.w, x.w[4] = v.x, x.w[5] = v.y, x.w[6] = v.z, x.w[7] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) x.w[e] = f[e];
        }
    }
    return x;
}

// The word of codes of 8 channels of a group (nibble e: x[e]) and the group's
// scale bits; the 4 lanes of a group are neighbours.
template <bool BF16>
__device__ __forceinline__ uint32_t quant_word(const Raw8 &raw, uint32_t *scale_bits)
{
    // the largest magnitude, as bits: those of infinities and NaN are larger than all others
    uint32_t top;
    float x[8];
    if (BF16) {
        top = __vmaxu2(__vmaxu2(raw.w[0] & 0x7fff7fffu, raw.w[1] & 0x7fff7fffu),
                       __vmaxu2(raw.w[2] & 0x7fff7fffu, raw.w[3] & 0x7fff7fffu));
        top = max(top & 0xffff0000u, top << 16);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            x[2 * e] = __uint_as_float(raw.w[e] << 16);
            x[2 * e + 1] = __uint_as_float(raw.w[e] & 0xffff0000u);
        }
    } else {
        top = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            top = max(top, raw.w[e] & 0x7fffffffu);
            x[e] = __uint_as_float(raw.w[e]);
        }
    }
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    const uint32_t sb = quant_scale_bits(__uint_as_float(top));
    *scale_bits = sb;
    const float s = bf16_bits_f32(sb);
    if (!(s > 0.0f)) return 0x88888888u;
    uint32_t word = 0;
    if (s >= 1e-18f) {
        // x inv + 1.5 2^23 + 8 rounds to the code in the low bits; codes are joined by adding those bits, shifted, and
        // taking the constant parts off.  |x| < 7.02 s, so no clamp; a value within rounding of a border is seen by
        // its remainder, which is exact (see quant_code)
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        constexpr float kMagic = 12582920.0f;
        uint32_t base = 0;
        float y[8], far = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            y[e] = fmaf(x[e], inv, kMagic);
            far = fmaxf(far, fabsf(fmaf(-(y[e] - kMagic), s, x[e])));
            word += __float_as_uint(y[e]) << (4 * e);
            base += 0x4b400000u << (4 * e);
        }
        word -= base;
        if (2.0f * far >= s) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float r = fmaf(-(y[e] - kMagic), s, x[e]), d = 2.0f * fabsf(r);
                if (d > s || (d == s && (__float_as_uint(y[e]) & 1u))) word += (r > 0.0f ? 1u : 0xffffffffu) << (4 * e);
            }
        }
        return word;
    }
    const float up = 18446744073709551616.0f;     // 2^64: 1 / s stays finite
    const float inv = __fdiv_rn(1.0f, s * up);
#pragma unroll
    for (int e = 0; e < 8; e++) word |= quant_code(x[e] * up, s * up, inv) << (4 * e);
    return word;
}

// Transpose of the 4 x 4 bytes of 4 neighbouring lanes' words: lane i gets
// byte i of lanes 0..3.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t w, int lane)
{
    uint32_t o = __shfl_xor_sync(kFull, w, 1);
    w = (lane & 1) ? __byte_perm(o, w, 0x7351) : __byte_perm(w, o, 0x6240);   // lanes 2i, 2i + 1: bytes (0, 0', 2, 2') and (1, 1', 3, 3')
    o = __shfl_xor_sync(kFull, w, 2);
    return (lane & 2) ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
}

// nibbles 0, 2, 4, 6 of a word of bytes 0x0n, and back
__device__ __forceinline__ uint32_t join_nibbles(uint32_t x)
{
    x = (x | x >> 4) & 0x00ff00ffu;
    return (x | x >> 8) & 0xffffu;
}
__device__ __forceinline__ uint32_t spread_nibbles(uint32_t x)
{
    x = (x | x << 8) & 0x00ff00ffu;
    return (x | x << 4) & 0x0f0f0f0fu;
}

// One CTA per 32-key block of the cache (or, of few rows, per pair).  A warp
// has rows 4w .. 4w + 3, two at a time: lane (row, group r, quarter t) has
// channels 32r + 8t .. + 7, whose codes are word (t, r) of a K row; of a V row
// they are nibble t of the 8 chunks, which the 4 lanes of a group exchange.
// The block is put together in shared memory and leaves by 16-byte stores.
template <bool BF16>
__global__ void __launch_bounds__(kQrThreads) k_quant_append(QuantRowsArgs a, int tiles)
{
    __shared__ __align__(16) uint8_t img[kQBlock];
    const int p = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const int64_t at = a.at ? a.at[p] : a.c.lens[p];
    const bool fits = at >= 0 && at + a.n_rows <= a.c.n_cap;
    const int r = (lane & 15) >> 2, t = lane & 3;
    for (int tile = blockIdx.x; fits && tile < tiles; tile += gridDim.x) {
        const int64_t b = at / kQKeys + tile, i0 = b * kQKeys - at;          // row of the block's first key
        if (i0 >= a.n_rows) break;
        const int j0 = (int)max((int64_t)0, -i0), j1 = (int)min((int64_t)kQKeys, a.n_rows - i0);
        if (4 * warp < j1 && 4 * warp + 4 > j0) {
            const int64_t base = ((int64_t)p * a.stride + i0) * kD + 8 * (lane & 15);
            Raw8 x[4];                   // K rows 4w + 2i + lane / 16, then V
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int j = 4 * warp + 2 * (i & 1) + (lane >> 4);
                x[i] = Raw8{};
                if (j >= j0 && j < j1) x[i] = load8<BF16>(i >> 1 ? a.v : a.k, base + (int64_t)j * kD, a.vec);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int j = 4 * warp + 2 * (i & 1) + (lane >> 4);
                uint32_t sb, w = quant_word<BF16>(x[i], &sb);
                if (i >> 1) {
                    w = transpose_bytes(w, lane);      // byte i: channels 8i + 2t, + 1 of the group
                    uint8_t *row = img + kQOffV + j * kQRow + 2 * r;
                    *reinterpret_cast<uint16_t *>(row + 8 * ((2 * t) ^ v_turn(j))) = (uint16_t)join_nibbles(w & 0x0f0f0f0fu);
                    *reinterpret_cast<uint16_t *>(row + 8 * ((2 * t + 1) ^ v_turn(j))) = (uint16_t)join_nibbles(w >> 4 & 0x0f0f0f0fu);
                } else {
                    *reinterpret_cast<uint32_t *>(img + j * kQRow + 16 * t + 4 * r) = w;
                }
                if (t == 0) *reinterpret_cast<uint16_t *>(img + (i >> 1 ? kQOffVs : kQOffKs) + 8 * j + 2 * r) = (uint16_t)sb;
            }
        }
        __syncthreads();
        uint8_t *dst = a.c.blocks + ((int64_t)p * (a.c.n_cap / kQKeys) + b) * kQBlock;
        const int o = tid & 127, off = tid >> 7 ? kQOffV : 0;
        if (o >= 4 * j0 && o < 4 * j1) reinterpret_cast<uint4 *>(dst + off)[o] = reinterpret_cast<const uint4 *>(img + off)[o];
        if (tid < 2 * kQKeys && (tid & 31) >= j0 && (tid & 31) < j1)
            reinterpret_cast<uint2 *>(dst + kQOffKs)[tid] = reinterpret_cast<const uint2 *>(img + kQOffKs)[tid];
        if (a.c.acc && tid >= j0 && tid < j1) a.c.acc[(int64_t)p * a.c.n_cap + b * kQKeys + tid] = 0.0f;
        if (gridDim.x < tiles) __syncthreads();
    }
    // the length may change once every CTA of the pair has read it: where one CTA does all, or the places are others'
    if (gridDim.x == 1 || a.own_at) {
        __syncthreads();
        if (blockIdx.x == 0 && tid == 0) {
            if (fits) a.c.lens[p] = (int32_t)(at + a.n_rows);
            else quant_devchk(a.c.status, p);
        }
    }
}

// New lengths after an append behind the lengths, of several CTAs per pair.
__global__ void k_quant_lens(QuantRowsArgs a)
{
    pdl_wait();
    const int p = blockIdx.x * blockDim.x + threadIdx.x;
    if (p >= a.c.bh) return;
    const int64_t at = a.at ? a.at[p] : a.c.lens[p];
    if (at >= 0 && at + a.n_rows <= a.c.n_cap) a.c.lens[p] = (int32_t)(at + a.n_rows);
    else quant_devchk(a.c.status, p);
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t i, const float x[8], int vec)
{
    if (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&h);
        }
        __nv_bfloat16 *d = reinterpret_cast<__nv_bfloat16 *>(p) + i;
        if (vec) {
            __stcs(reinterpret_cast<uint4 *>(d), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) reinterpret_cast<uint16_t *>(d)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    } else {
        float *d = reinterpret_cast<float *>(p) + i;
        if (vec) {
            __stcs(reinterpret_cast<float4 *>(d), make_float4(x[0], x[1], x[2], x[3]));
            __stcs(reinterpret_cast<float4 *>(d) + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) d[e] = x[e];
        }
    }
}

// Append the other way round: one CTA per block.
template <bool BF16>
__global__ void __launch_bounds__(kQrThreads) k_quant_rows(QuantRowsArgs a)
{
    __shared__ __align__(16) uint8_t img[kQBlock];
    const int p = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const int64_t at = a.at ? a.at[p] : 0;
    const int n = quant_len(a.c, p);
    if (blockIdx.x == 0 && tid == 0 && quant_len_bad(a.c, p)) quant_devchk(a.c.status, p);
    const int64_t b = max(at, (int64_t)0) / kQKeys + blockIdx.x;
    const int64_t i0 = b * kQKeys - at;          // row of the block's first key
    const int j0 = (int)max((int64_t)0, -i0);
    const int j1 = (int)max((int64_t)0, min(min((int64_t)kQKeys, a.n_rows - i0), n - b * kQKeys));
    if (j0 >= j1) return;
    const uint8_t *src = a.c.blocks + ((int64_t)p * (a.c.n_cap / kQKeys) + b) * kQBlock;
    reinterpret_cast<uint4 *>(img)[tid] = __ldcs(reinterpret_cast<const uint4 *>(src) + tid);
    if (tid < kQBlock / 16 - kQrThreads) reinterpret_cast<uint4 *>(img)[kQrThreads + tid] = __ldcs(reinterpret_cast<const uint4 *>(src) + kQrThreads + tid);
    __syncthreads();
    const int r = (lane & 15) >> 2, t = lane & 3;
    const int64_t base = ((int64_t)p * a.stride + i0) * kD + 8 * (lane & 15);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int j = 4 * warp + 2 * (i & 1) + (lane >> 4);
        uint32_t w;
        if (i >> 1) {
            const uint8_t *row = img + kQOffV + j * kQRow + 2 * r;
            const uint32_t e = *reinterpret_cast<const uint16_t *>(row + 8 * ((2 * t) ^ v_turn(j)));
            const uint32_t o = *reinterpret_cast<const uint16_t *>(row + 8 * ((2 * t + 1) ^ v_turn(j)));
            w = transpose_bytes(spread_nibbles(e) | spread_nibbles(o) << 4, lane);
        } else {
            w = *reinterpret_cast<const uint32_t *>(img + j * kQRow + 16 * t + 4 * r);
        }
        if (j < j0 || j >= j1) continue;
        const float s = bf16_bits_f32(*reinterpret_cast<const uint16_t *>(img + (i >> 1 ? kQOffVs : kQOffKs) + 8 * j + 2 * r));
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = ((float)((w >> (4 * e)) & 15u) - 8.0f) * s;
        store8<BF16>(const_cast<void *>(i >> 1 ? a.v : a.k), base + (int64_t)j * kD, x, a.vec);
    }
}

// blocks that n rows can touch, from any place on
static int row_tiles(int64_t n) { return (int)((n + 2 * kQKeys - 2) / kQKeys); }

cudaError_t launch_quant_append(const QuantRowsArgs &a, cudaStream_t s)
{
    // up to 4 blocks a pair: one CTA does them in turn and sets the length; a second launch would cost more
    const int tiles = row_tiles(a.n_rows), ctas = tiles <= 4 ? 1 : tiles;
    cudaError_t e = launch_pdl(a.is_bf16 ? k_quant_append<true> : k_quant_append<false>, dim3(ctas, a.c.bh), dim3(kQrThreads), 0, s, a, tiles);
    if (e == cudaSuccess && ctas > 1 && !a.own_at)
        e = launch_pdl(k_quant_lens, dim3((a.c.bh + 255) / 256), dim3(256), 0, s, a);
    return e;
}

cudaError_t launch_quant_rows(const QuantRowsArgs &a, cudaStream_t s)
{
    return launch_pdl(a.is_bf16 ? k_quant_rows<true> : k_quant_rows<false>, dim3(row_tiles(a.n_rows), a.c.bh), dim3(kQrThreads), 0, s, a);
}

}  // namespace pk
