// pk_quant.cu -- host side of the 4-bit KV cache calls (pk_quant_*): argument
// checks and launches.  Nothing is allocated and no state is kept.
#include <cmath>

#include "pk_quant.cuh"

using namespace pk;

namespace {

// Device memory of the current device, or (unless `device_only`) page-locked /
// managed host memory.
bool quant_accessible(const void *ptr, size_t align, bool device_only = false)
{
    cudaPointerAttributes at;
    if (!ptr || ((uintptr_t)ptr % align) != 0) return false;
    if (cudaPointerGetAttributes(&at, ptr) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (at.type == cudaMemoryTypeDevice) {
        int dev = -1;
        return cudaGetDevice(&dev) == cudaSuccess && at.device == dev;
    }
    return !device_only && (at.type == cudaMemoryTypeHost || at.type == cudaMemoryTypeManaged);
}

pk_status quant_status(cudaError_t e)
{
    if (e == cudaSuccess) return PK_OK;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? PK_ERR_OOM : PK_ERR_CUDA;
}

pk_status check_sizes(const pk_quant_cache *c)
{
    if (!c || c->bh < 1) return PK_ERR_INVALID_ARG;
    if (c->bh > 65535) return PK_ERR_UNSUPPORTED;
    if (c->kv_dtype != PK_F32 && c->kv_dtype != PK_BF16) return PK_ERR_INVALID_ARG;
    if (c->n_cap < kQKeys || c->n_cap % kQKeys != 0) return PK_ERR_INVALID_ARG;
    if (c->n_cap > (int64_t)0x7fffffff - kQKeys) return PK_ERR_CAPACITY;
    return PK_OK;
}

pk_status check_cache(const pk_quant_cache *c, QuantCache *out)
{
    const pk_status st = check_sizes(c);
    if (st != PK_OK) return st;
    if (!quant_accessible(c->blocks, 16, true) || !quant_accessible(c->lens, 4, true)) return PK_ERR_INVALID_ARG;
    if (c->acc && !quant_accessible(c->acc, 4, true)) return PK_ERR_INVALID_ARG;
    if (c->status && !quant_accessible(c->status, 4, true)) return PK_ERR_INVALID_ARG;
    *out = QuantCache{(uint8_t *)c->blocks, c->lens, c->acc, c->status, c->n_cap, c->bh};
    return PK_OK;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// bytes on whose boundary two arrays' rows lie
int32_t row_boundary(const void *a, const void *b)
{
    const uintptr_t x = (uintptr_t)a | (uintptr_t)b;
    return x % 32 == 0 ? 32 : x % 16 == 0 ? 16 : 0;
}

// bytes of the partial results, a multiple of 256
size_t part_bytes(int32_t bh, int32_t G)
{
    const size_t n = ((size_t)bh + kQMaxWorkers) * G * kQPart * sizeof(float);
    return (n + 255) / 256 * 256;
}

// bytes of the table of partial results, a multiple of 256
size_t parts_bytes(int32_t bh) { return ((size_t)bh * sizeof(uint2) + 255) / 256 * 256; }

}  // namespace

extern "C" {

pk_status pk_quant_append(const pk_quant_cache *cache, const void *k_new, const void *v_new, int64_t n_new,
                          int64_t src_stride, const int32_t *at, void *stream)
{
    QuantRowsArgs a{};
    const pk_status st = check_cache(cache, &a.c);
    if (st != PK_OK) return st;
    if (n_new < 1 || src_stride < 0 || (src_stride != 0 && src_stride < n_new)) return PK_ERR_INVALID_ARG;
    if (n_new > cache->n_cap) return PK_ERR_CAPACITY;
    const size_t es = cache->kv_dtype == PK_BF16 ? 2 : 4;
    if (!quant_accessible(k_new, es) || !quant_accessible(v_new, es) || (at && !quant_accessible(at, 4)))
        return PK_ERR_INVALID_ARG;
    const bool meets = at && overlap(at, (size_t)cache->bh * 4, cache->lens, (size_t)cache->bh * 4);
    if (meets && at != cache->lens) return PK_ERR_INVALID_ARG;       // one pair's place, another's length
    a.k = k_new;
    a.v = v_new;
    a.n_rows = n_new;
    a.stride = src_stride ? src_stride : n_new;
    a.at = at;
    a.own_at = at && !meets;
    a.is_bf16 = cache->kv_dtype == PK_BF16;
    a.vec = row_boundary(k_new, v_new);
    return quant_status(launch_quant_append(a, (cudaStream_t)stream));
}

pk_status pk_quant_rows(const pk_quant_cache *cache, int64_t n_rows, void *k_out, void *v_out, const int32_t *at,
                        void *stream)
{
    QuantRowsArgs a{};
    const pk_status st = check_cache(cache, &a.c);
    if (st != PK_OK) return st;
    if (n_rows < 1 || n_rows > 0x7fffffff) return PK_ERR_INVALID_ARG;
    const size_t es = cache->kv_dtype == PK_BF16 ? 2 : 4;
    if (!quant_accessible(k_out, es) || !quant_accessible(v_out, es) || (at && !quant_accessible(at, 4)))
        return PK_ERR_INVALID_ARG;
    a.k = k_out;
    a.v = v_out;
    a.n_rows = n_rows;
    a.stride = n_rows;
    a.at = at;
    a.is_bf16 = cache->kv_dtype == PK_BF16;
    a.vec = row_boundary(k_out, v_out);
    return quant_status(launch_quant_rows(a, (cudaStream_t)stream));
}

pk_status pk_quant_attend_workspace(const pk_quant_cache *cache, int32_t group, int32_t accumulate, size_t *bytes)
{
    const pk_status st = check_sizes(cache);
    if (st != PK_OK) return st;
    if (!bytes || group < 1 || group > kMaxGroup) return PK_ERR_INVALID_ARG;
    *bytes = part_bytes(cache->bh, group) + parts_bytes(cache->bh);
    if (accumulate) *bytes += (size_t)cache->bh * group * (size_t)cache->n_cap * sizeof(float);
    return PK_OK;
}

pk_status pk_quant_attend(const pk_quant_cache *cache, const void *q, int32_t group, float scale, float *out,
                          float *lse, int32_t accumulate, void *work, size_t work_bytes, void *stream)
{
    QuantAttendArgs a{};
    pk_status st = check_cache(cache, &a.c);
    if (st != PK_OK) return st;
    size_t need = 0;
    st = pk_quant_attend_workspace(cache, group, accumulate, &need);
    if (st != PK_OK) return st;
    if (!(scale >= 0.0f) || std::isinf(scale) || (accumulate && !cache->acc)) return PK_ERR_INVALID_ARG;
    if (!quant_accessible(q, cache->kv_dtype == PK_BF16 ? 2 : 4) || !quant_accessible(out, 4) ||
        (lse && !quant_accessible(lse, 4)) || !quant_accessible(work, 256, true))
        return PK_ERR_INVALID_ARG;
    if (work_bytes < need) return PK_ERR_CAPACITY;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return quant_status(e);
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.part = (float *)work;
    a.parts = (uint2 *)((char *)work + part_bytes(cache->bh, group));
    a.logits = accumulate ? (float *)((char *)a.parts + parts_bytes(cache->bh)) : nullptr;
    a.G = group;
    a.is_bf16 = cache->kv_dtype == PK_BF16;
    a.accumulate = accumulate != 0;
    const double s = scale > 0.0f ? (double)scale : 1.0 / std::sqrt((double)kD);
    a.scale2 = (float)(s * 1.4426950408889634074);
    return quant_status(launch_quant_attend(a, sms, (cudaStream_t)stream));
}

pk_status pk_quant_evict(const pk_quant_cache *src, const pk_quant_cache *dst, int64_t budget, int64_t sink,
                         int64_t recent, int32_t *keep, void *stream)
{
    QuantEvictArgs a{};
    pk_status st = check_cache(src, &a.src);
    if (st == PK_OK) st = check_cache(dst, &a.dst);
    if (st != PK_OK) return st;
    if (!src->acc || src->bh != dst->bh || src->kv_dtype != dst->kv_dtype) return PK_ERR_INVALID_ARG;
    if (budget < 1 || sink < 0 || recent < 0 || sink > budget || recent > budget - sink) return PK_ERR_INVALID_ARG;
    if (dst->n_cap < (budget < src->n_cap ? budget : src->n_cap)) return PK_ERR_CAPACITY;
    if (budget > 0x7fffffff) return PK_ERR_CAPACITY;
    if (keep && !quant_accessible(keep, 4)) return PK_ERR_INVALID_ARG;
    const size_t ns = (size_t)src->bh * (src->n_cap / kQKeys) * kQBlock, nd = (size_t)dst->bh * (dst->n_cap / kQKeys) * kQBlock;
    const size_t ws = (size_t)src->bh * src->n_cap * 4, wd = (size_t)dst->bh * dst->n_cap * 4;
    if (overlap(src->blocks, ns, dst->blocks, nd) || overlap(src->lens, (size_t)src->bh * 4, dst->lens, (size_t)dst->bh * 4) ||
        (dst->acc && overlap(src->acc, ws, dst->acc, wd)))
        return PK_ERR_INVALID_ARG;
    const size_t nk = (size_t)src->bh * (size_t)budget * 4;
    if (keep && (overlap(keep, nk, src->blocks, ns) || overlap(keep, nk, dst->blocks, nd) || overlap(keep, nk, src->acc, ws) ||
                 (dst->acc && overlap(keep, nk, dst->acc, wd)) || overlap(keep, nk, src->lens, (size_t)src->bh * 4) ||
                 overlap(keep, nk, dst->lens, (size_t)dst->bh * 4)))
        return PK_ERR_INVALID_ARG;       // the kept rows' list, read while the others are written
    a.budget = budget;
    a.sink = sink;
    a.recent = recent;
    a.keep = keep;
    return quant_status(launch_quant_evict(a, (cudaStream_t)stream));
}

}  // extern "C"
