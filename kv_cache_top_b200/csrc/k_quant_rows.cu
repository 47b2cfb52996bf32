// k_quant_rows.cu -- rows into and out of the 4-bit KV cache.
//
// Append: scale_r = bf16(max|x| / 7) over a group of 32 channels, code = 8 +
// round(x / scale) (ties to even, clamped to -7..7).  Reads 2 D es bytes per
// key and writes 144; read-back the other way round.  Both are bound by
// memory: 32768 bf16 rows of 8 pairs are appended and read back in 59 us, 52 at
// the rate of a copy.
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

// the 32 channels of a group
template <bool BF16>
__device__ __forceinline__ void load_group(Raw8 x[4], const void *p, int64_t i, int vec)
{
    if (vec < 32) {
#pragma unroll
        for (int c = 0; c < 4; c++) x[c] = load8<BF16>(p, i + 8 * c, vec);
        return;
    }
    // 32 bytes at once: by 16 each sector would be asked for twice (32768 rows of 8 pairs: 30 us alone, 37)
    const uint8_t *b = reinterpret_cast<const uint8_t *>(p) + i * (BF16 ? 2 : 4);
#pragma unroll
    for (int c = 0; c < (BF16 ? 2 : 4); c++) {
        uint32_t w[8];
        asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(b + 32 * c)
                     : "memory");
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if (BF16) x[2 * c + e / 4].w[e % 4] = w[e];
            else x[c].w[e] = w[e];
        }
    }
}

// The codes of a group's 32 channels (x[i].. : channels 8i .. 8i + 7) and its
// scale bits.  K: word i has channels 8i + e as nibbles e; V: word e / 2 has
// channels 8i + e as nibbles 4 (e % 2) + i.
template <bool BF16, bool VALUES>
__device__ __forceinline__ void quant_group(const Raw8 raw[4], uint32_t word[4], uint32_t *scale_bits)
{
    // the largest magnitude, as bits: those of infinities and NaN are larger than all others
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int e = 0; e < (BF16 ? 4 : 8); e++)
            top = BF16 ? __vmaxu2(top, raw[i].w[e] & 0x7fff7fffu) : max(top, raw[i].w[e] & 0x7fffffffu);
    if (BF16) top = max(top & 0xffff0000u, top << 16);
    const uint32_t sb = quant_scale_bits(__uint_as_float(top));
    *scale_bits = sb;
    const float s = bf16_bits_f32(sb);
    auto pair = [&](int i, int h) {      // channels 8i + 2h, + 1
        return BF16 ? make_float2(__uint_as_float(raw[i].w[h] << 16), __uint_as_float(raw[i].w[h] & 0xffff0000u))
                    : make_float2(__uint_as_float(raw[i].w[2 * h]), __uint_as_float(raw[i].w[2 * h + 1]));
    };
    auto place = [&](int i, int e, uint32_t code) {      // or a difference to a code
        word[VALUES ? e >> 1 : i] += code << (VALUES ? 16 * (e & 1) + 4 * i : 4 * e);
    };
    if (!(s > 0.0f)) {
#pragma unroll
        for (int i = 0; i < 4; i++) word[i] = 0x88888888u;
        return;
    }
    if (s < 1e-18f) {
        const float up = 18446744073709551616.0f;     // 2^64: 1 / s stays finite
        const float inv = __fdiv_rn(1.0f, s * up);
#pragma unroll
        for (int i = 0; i < 4; i++) word[i] = 0;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int h = 0; h < 4; h++) {
                const float2 x = pair(i, h);
                place(i, 2 * h, quant_code(x.x * up, s * up, inv));
                place(i, 2 * h + 1, quant_code(x.y * up, s * up, inv));
            }
        return;
    }
    // x inv + 1.5 2^23 + 8 rounds to the code in the low bits; codes are joined by adding those bits, shifted, and
    // taking the constant parts off.  |x| < 7.02 s, so no clamp
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    constexpr float kMagic = 12582920.0f;
    uint32_t base = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) base += 0x4b400000u << (4 * e);
#pragma unroll
    for (int i = 0; i < 4; i++) word[i] = 0u - base;
    if (BF16) {
        // |x / s - (k + 1/2)| = |2 x - (2 k + 1) s| / 2 s is 0 or at least 2^-10: 2 x is a multiple of half a unit of s
        // from |x| = s / 4 on.  So x inv (off by 2^-19) is rounded to a multiple of 2^-11 first, which makes ties exact
        // and moves nothing over a border
        constexpr float kSnap = 6144.0f;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int h = 0; h < 4; h++) {
                const float2 y = add2(fma2(pair(i, h), make_float2(inv, inv), make_float2(kSnap, kSnap)),
                                      make_float2(kMagic - kSnap, kMagic - kSnap));
                place(i, 2 * h, __float_as_uint(y.x));
                place(i, 2 * h + 1, __float_as_uint(y.y));
            }
        return;
    }
    // a value within rounding of a border is seen by its remainder, which is exact (see quant_code)
    auto code = [&](float2 x) { return fma2(x, make_float2(inv, inv), make_float2(kMagic, kMagic)); };
    auto rest = [&](float2 x, float2 y) { return fma2(add2(y, make_float2(-kMagic, -kMagic)), make_float2(-s, -s), x); };
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int h = 0; h < 4; h++) {
            const float2 x = pair(i, h), y = code(x), r = rest(x, y);
            far = fmaxf(far, fmaxf(fabsf(r.x), fabsf(r.y)));
            place(i, 2 * h, __float_as_uint(y.x));
            place(i, 2 * h + 1, __float_as_uint(y.y));
        }
    if (2.0f * far < s) return;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int h = 0; h < 4; h++) {
            const float2 x = pair(i, h), y = code(x), r = rest(x, y);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float re = e ? r.y : r.x, d = 2.0f * fabsf(re);
                if (d > s || (d == s && (__float_as_uint(e ? y.y : y.x) & 1u))) place(i, 2 * h + e, re > 0.0f ? 1u : 0xffffffffu);
            }
        }
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

// nibbles 0..3 as the bytes 0x0n of a word
__device__ __forceinline__ uint32_t spread_nibbles(uint32_t x)
{
    x = (x | x << 8) & 0x00ff00ffu;
    return (x | x << 4) & 0x0f0f0f0fu;
}

// One CTA per 32-key block of the cache (or, of few rows, per pair).  A thread
// has a group of 32 channels of a row of K or V: what a group needs once (the
// scale) is then computed once, and codes are put in place without a shuffle.
// The block is put together in shared memory and leaves by 16-byte stores.
// bf16: 40 registers, 6 CTAs to an SM (65 us with the read-back, 68 at 4 to an
// SM); fp32 needs 79.
template <bool BF16>
__global__ void __launch_bounds__(kQrThreads, BF16 ? 6 : 3) k_quant_append(QuantRowsArgs a, int tiles)
{
    // rows 80 bytes apart: the stores of 8 rows meet in fewer banks
    __shared__ __align__(16) uint8_t img[2][kQKeys][kQRow + 16];
    __shared__ __align__(16) uint16_t scale[2][kQKeys][4];
    const int p = blockIdx.y, tid = threadIdx.x;
    pdl_wait();
    const int64_t at = a.at ? a.at[p] : a.c.lens[p];
    const bool fits = at >= 0 && at + a.n_rows <= a.c.n_cap;
    const int j = tid >> 2 & 31, r = tid & 3;
    for (int tile = blockIdx.x; fits && tile < tiles; tile += gridDim.x) {
        const int64_t b = at / kQKeys + tile, i0 = b * kQKeys - at;          // row of the block's first key
        if (i0 >= a.n_rows) break;
        const int j0 = (int)max((int64_t)0, -i0), j1 = (int)min((int64_t)kQKeys, a.n_rows - i0);
        if (j >= j0 && j < j1) {
            const int64_t base = ((int64_t)p * a.stride + i0 + j) * kD + 32 * r;
            const bool values = tid >= 4 * kQKeys;
            Raw8 x[4];
            uint32_t w[4], sb;
            load_group<BF16>(x, values ? a.v : a.k, base, a.vec);
            if (values) {
                quant_group<BF16, true>(x, w, &sb);
                uint8_t *row = img[1][j] + 2 * r;
#pragma unroll
                for (int g = 0; g < 8; g++) *reinterpret_cast<uint16_t *>(row + 8 * (g ^ v_turn(j))) = (uint16_t)(w[g >> 1] >> (16 * (g & 1)));
            } else {
                quant_group<BF16, false>(x, w, &sb);
#pragma unroll
                for (int i = 0; i < 4; i++) *reinterpret_cast<uint32_t *>(img[0][j] + 16 * i + 4 * r) = w[i];
            }
            scale[values][j][r] = (uint16_t)sb;
        }
        __syncthreads();
        uint8_t *dst = a.c.blocks + ((int64_t)p * (a.c.n_cap / kQKeys) + b) * kQBlock;
        if (j >= j0 && j < j1) reinterpret_cast<uint4 *>(dst + (tid >> 7 ? kQOffV : 0))[tid & 127] = reinterpret_cast<const uint4 *>(img[tid >> 7][j])[r];
        if (tid < 2 * kQKeys && (tid & 31) >= j0 && (tid & 31) < j1)
            reinterpret_cast<uint2 *>(dst + kQOffKs)[tid] = reinterpret_cast<const uint2 *>(scale)[tid];
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

// Append the other way round: one CTA per kQrBlocks blocks, whose bytes are on
// their way at once (32768 rows of 8 pairs, append included: 59 us for 65; of
// 15 pairs of 2001 rows 0.5 us more).
constexpr int kQrBlocks = 2;
template <bool BF16>
__global__ void __launch_bounds__(kQrThreads) k_quant_rows(QuantRowsArgs a)
{
    __shared__ __align__(16) uint8_t imgs[kQrBlocks][kQBlock];
    const int p = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const int64_t at = a.at ? a.at[p] : 0;
    const int n = quant_len(a.c, p);
    if (blockIdx.x == 0 && tid == 0 && quant_len_bad(a.c, p)) quant_devchk(a.c.status, p);
    const int64_t b0 = max(at, (int64_t)0) / kQKeys + (int64_t)blockIdx.x * kQrBlocks;
    const int64_t end = min(at + a.n_rows, (int64_t)n);          // slots behind the last
    const uint8_t *src = a.c.blocks + ((int64_t)p * (a.c.n_cap / kQKeys) + b0) * kQBlock;
    const int blocks = (int)max((int64_t)0, min((int64_t)kQrBlocks, (end + kQKeys - 1) / kQKeys - b0));
    constexpr int kPer = (kQrBlocks * kQBlock / 16 + kQrThreads - 1) / kQrThreads;
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (i * kQrThreads + tid < blocks * (kQBlock / 16)) v[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i * kQrThreads + tid);
#pragma unroll
    for (int i = 0; i < kPer; i++)
        if (i * kQrThreads + tid < blocks * (kQBlock / 16)) reinterpret_cast<uint4 *>(imgs)[i * kQrThreads + tid] = v[i];
    __syncthreads();
    const int r = (lane & 15) >> 2, t = lane & 3;
#pragma unroll 1
    for (int y = 0; y < blocks; y++) {
        const uint8_t *img = imgs[y];
        const int64_t b = b0 + y, i0 = b * kQKeys - at;          // row of the block's first key
        const int j0 = (int)max((int64_t)0, -i0), j1 = (int)min((int64_t)kQKeys, end - b * kQKeys);
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
    return launch_pdl(a.is_bf16 ? k_quant_rows<true> : k_quant_rows<false>, dim3((row_tiles(a.n_rows) + kQrBlocks - 1) / kQrBlocks, a.c.bh), dim3(kQrThreads), 0, s, a);
}

}  // namespace pk
