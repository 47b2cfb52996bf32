// k_quant_attend.cu -- softmax attention over the 4-bit KV cache.
//
// z_gj = scale <q_g, K_j>, out_g = sum_j softmax(z_g)_j V_j, with an online
// softmax per worker's segment of a pair and a merge of the segments; when
// weights are accumulated, the logits go to the workspace and the merge
// kernel, which knows each head's log-sum, adds the weights to acc.
#include "pk_launch.cuh"
#include "pk_quant.cuh"

namespace pk {

constexpr int kQaThreads = 128;
constexpr int kQaMinShare = 8;           // blocks a worker takes at least
constexpr int kQmThreads = 256;          // merge kernel
constexpr int kQmKeys = 2048;            // keys of a merge CTA's part of acc

int quant_attend_workers(int num_sms) { return min(4 * num_sms, kQMaxWorkers); }

__device__ __forceinline__ int64_t block_count(const QuantCache &c, int p) { return (quant_len(c, p) + kQKeys - 1) / kQKeys; }

// Sum of the block counts of pairs [0, end) over a CTA of NT threads.
template <int NT>
__device__ int64_t count_blocks(const QuantCache &c, int end, long long *s)
{
    long long v = 0;
    for (int p = threadIdx.x; p < end; p += NT) v += block_count(c, p);
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < NT / 32; w++) v += s[w];
    __syncthreads();
    return v;
}

__global__ void __launch_bounds__(kQaThreads) k_quant_attend(QuantAttendArgs a)
{
    __shared__ float s_q[kMaxGroup][kD];
    __shared__ float s_kv[kQKeys][kD + 1];
    __shared__ float s_p[kMaxGroup][kQKeys];
    __shared__ float s_m[kMaxGroup], s_l[kMaxGroup], s_c[kMaxGroup];
    __shared__ long long s_sum[kQaThreads / 32];
    const int tid = threadIdx.x, w = blockIdx.x, G = a.G;
    pdl_wait();
    pdl_trigger();
    const int64_t total = count_blocks<kQaThreads>(a.c, a.c.bh, s_sum);
    const int64_t share = quant_share(total, a.workers, kQaMinShare);
    int64_t x = w * share;
    const int64_t end = min(total, x + share);
    if (x >= end) return;
    int p = 0;
    int64_t first = 0;                   // first block of pair p in the total
    while (first + block_count(a.c, p) <= x) first += block_count(a.c, p++);
    for (; x < end; p++) {
        const int64_t nb = block_count(a.c, p);
        const int n = quant_len(a.c, p);
        const int64_t b0 = x - first, b1 = min(nb, end - first);
        first += nb;
        if (b0 >= b1) continue;
        x += b1 - b0;
        __syncthreads();
        for (int i = tid; i < G * kD; i += kQaThreads) s_q[i / kD][i % kD] = ld_as_f32(a.q, (int64_t)p * G * kD + i, a.is_bf16);
        if (tid < kMaxGroup) {
            s_m[tid] = -INFINITY;
            s_l[tid] = 0.0f;
        }
        float acc[kMaxGroup];
#pragma unroll
        for (int g = 0; g < kMaxGroup; g++) acc[g] = 0.0f;
        for (int64_t b = b0; b < b1; b++) {
            const uint8_t *blk = a.c.blocks + ((int64_t)p * (a.c.n_cap / kQKeys) + b) * kQBlock;
            const int valid = (int)min((int64_t)kQKeys, n - b * kQKeys);
            __syncthreads();
            const int c = tid, r = c >> 5, t = (c & 31) >> 3, i = c & 7;
            for (int j = 0; j < kQKeys; j++) {
                const int nib = 32 * t + 8 * r + i;
                const float s = bf16_bits_f32(reinterpret_cast<const uint16_t *>(blk + kQOffKs)[4 * j + r]);
                s_kv[j][c] = j < valid ? (float)((blk[j * kQRow + nib / 2] >> (4 * (nib & 1)) & 15) - 8) * s : 0.0f;
            }
            __syncthreads();
            for (int e = tid; e < G * kQKeys; e += kQaThreads) {
                const int g = e / kQKeys, j = e % kQKeys;
                float z = 0.0f;
                for (int d = 0; d < kD; d++) z = fmaf(s_q[g][d], s_kv[j][d], z);
                z *= a.scale2;
                s_p[g][j] = j < valid ? z : -INFINITY;
                if (a.logits) a.logits[(((int64_t)p * (a.c.n_cap / kQKeys) + b) * G + g) * kQKeys + j] = z;
            }
            __syncthreads();
            if (tid < G) {
                float m = s_m[tid];
                for (int j = 0; j < kQKeys; j++) m = fmaxf(m, s_p[tid][j]);
                const float ref = m == -INFINITY ? 0.0f : m;
                s_c[tid] = exp2f(s_m[tid] - ref);
                float l = s_l[tid] * s_c[tid];
                for (int j = 0; j < kQKeys; j++) l += s_p[tid][j] = exp2f(s_p[tid][j] - ref);
                s_l[tid] = l;
                s_m[tid] = m;
            }
            for (int j = 0; j < kQKeys; j++) {
                const int nib = 16 * (i ^ v_turn(j)) + 4 * r + t;      // channel 32 r + 8 t + i
                const float s = bf16_bits_f32(reinterpret_cast<const uint16_t *>(blk + kQOffVs)[4 * j + r]);
                s_kv[j][c] = j < valid ? (float)((blk[kQOffV + j * kQRow + nib / 2] >> (4 * (nib & 1)) & 15) - 8) * s : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kMaxGroup; g++) {
                if (g >= G) break;
                float o = acc[g] * s_c[g];
                for (int j = 0; j < valid; j++) o = fmaf(s_p[g][j], s_kv[j][tid], o);
                acc[g] = o;
            }
        }
        float *part = a.part + (int64_t)(p + w) * G * kQPart;
        __syncthreads();
#pragma unroll
        for (int g = 0; g < kMaxGroup; g++) {
            if (g >= G) break;
            part[g * kQPart + tid] = acc[g];
            if (tid == 0) {
                part[g * kQPart + kD] = s_m[g];
                part[g * kQPart + kD + 1] = s_l[g];
            }
        }
    }
}

// Merge of a pair's partial results (CTAs x < G: head x) and its part of acc
// (CTAs x >= G: keys [(x - G) kQmKeys, ...)).
__global__ void __launch_bounds__(kQmThreads) k_quant_merge(QuantAttendArgs a)
{
    __shared__ long long s_sum[kQmThreads / 32];
    __shared__ float s_lse[kMaxGroup];
    const int tid = threadIdx.x, p = blockIdx.y, G = a.G;
    pdl_wait();
    const int n = quant_len(a.c, p);
    const bool is_out = (int)blockIdx.x < G;
    const int64_t k0 = (int64_t)((int)blockIdx.x - G) * kQmKeys;
    if (!is_out && k0 >= n) return;
    if (is_out && blockIdx.x == 0 && tid == 0 && quant_len_bad(a.c, p)) quant_devchk(a.c.status, p);
    if (n == 0) {
        if (tid < kD) a.out[((int64_t)p * G + blockIdx.x) * kD + tid] = 0.0f;
        if (tid == 0 && a.lse) a.lse[(int64_t)p * G + blockIdx.x] = -INFINITY;
        return;
    }
    const int64_t total = count_blocks<kQmThreads>(a.c, a.c.bh, s_sum);
    const int64_t first = count_blocks<kQmThreads>(a.c, p, s_sum);
    const int64_t share = quant_share(total, a.workers, kQaMinShare);
    const int w0 = (int)(first / share), w1 = (int)((first + block_count(a.c, p) - 1) / share);
    const float *part = a.part + (int64_t)(p + w0) * G * kQPart;
    const int ns = w1 - w0 + 1;
    const int warp = tid >> 5, lane = tid & 31;
    for (int g = is_out ? blockIdx.x : warp; g < G; g += is_out ? G : kQmThreads / 32) {
        const float *pg = part + (int64_t)g * kQPart + kD;
        float m = -INFINITY;
        for (int s = lane; s < ns; s += 32) m = fmaxf(m, pg[(int64_t)s * G * kQPart]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        const float ref = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
        for (int s = lane; s < ns; s += 32) l += exp2f(pg[(int64_t)s * G * kQPart] - ref) * pg[(int64_t)s * G * kQPart + 1];
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
        if (is_out) {
            if (tid < kD) {
                float o = 0.0f;
                for (int s = 0; s < ns; s++)
                    o = fmaf(exp2f(pg[(int64_t)s * G * kQPart] - ref), pg[(int64_t)s * G * kQPart - kD + tid], o);
                a.out[((int64_t)p * G + g) * kD + tid] = l == 0.0f ? 0.0f : o / l;
            }
            if (tid == 0 && a.lse) a.lse[(int64_t)p * G + g] = (log2f(l) + ref) * 0.69314718055994531f;
        } else if (lane == 0) {
            s_lse[g] = l == 0.0f ? INFINITY : log2f(l) + ref;
        }
    }
    if (is_out) return;
    __syncthreads();
    for (int64_t k = k0 + tid; k < min((int64_t)n, k0 + kQmKeys); k += kQmThreads) {
        const float *z = a.logits + ((int64_t)p * (a.c.n_cap / kQKeys) + k / kQKeys) * G * kQKeys + k % kQKeys;
        float sum = 0.0f;
        for (int g = 0; g < G; g++) sum += exp2f(z[g * kQKeys] - s_lse[g]);
        a.c.acc[(int64_t)p * a.c.n_cap + k] += sum;
    }
}

cudaError_t launch_quant_attend(const QuantAttendArgs &a, cudaStream_t s)
{
    cudaError_t e = launch_pdl(k_quant_attend, dim3(a.workers), dim3(kQaThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const unsigned parts = a.accumulate ? (unsigned)((a.c.n_cap + kQmKeys - 1) / kQmKeys) : 0u;
    return launch_pdl(k_quant_merge, dim3(a.G + parts, a.c.bh), dim3(kQmThreads), 0, s, a);
}

}  // namespace pk
