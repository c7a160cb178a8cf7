// C ABI of the operators around the search: argument checks, the handles of the output
// layer and its adapters, and the launches. Every call is asynchronous on the caller's stream
// unless its declaration says otherwise, keeps the calling thread's current
// device, and lets no exception out.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <new>
#include <string>

#include "wfst.h"
#include "wfst_score.h"

using namespace wfst;

struct wfst_layer_s {
    int device = -1;
    void *block = nullptr;       // one allocation: weights, scales, zeros, bias
    Layer l{};
};

struct wfst_adapters_s {
    int device = -1;
    void *block = nullptr;       // one allocation: down, up, scales, ranks
    Adapters a{};
};

namespace {

int hip_fail(hipError_t e, const char *what)
{
    (void)hipGetLastError();     // (a later call's launch must not report this one's error)
    return api_fail(e == hipErrorOutOfMemory ? WFST_ENOMEM : WFST_EDEVICE,
                    std::string(what) + ": " + hipGetErrorString(e));
}

#define HIP_TRY(expr)                                              \
    do {                                                           \
        hipError_t _e = (expr);                                    \
        if (_e != hipSuccess) return hip_fail(_e, #expr);          \
    } while (0)

// Makes `device` current for a call and restores the caller's device after it.
class DeviceScope {
public:
    hipError_t enter(int device)
    {
        hipError_t e = hipGetDevice(&old_);
        if (e != hipSuccess) return e;
        if (old_ == device) return hipSuccess;
        e = hipSetDevice(device);
        changed_ = e == hipSuccess;
        return e;
    }
    ~DeviceScope()
    {
        if (changed_) (void)hipSetDevice(old_);
    }

private:
    int old_ = 0;
    bool changed_ = false;
};

template <typename F>
int guarded(F &&f)
{
    try {
        return f();
    } catch (const std::bad_alloc &) {
        return WFST_ENOMEM;
    } catch (...) {
        return WFST_EDEVICE;
    }
}

bool dtype_ok(int32_t t) { return t == WFST_LP_F32 || t == WFST_LP_F16 || t == WFST_LP_BF16; }

// Bytes from the first to past the last element of `rows` rows of n elements
// `stride` elements apart; -1 when that passes 2^62.
int64_t span_bytes(int64_t rows, int64_t n, int64_t stride, size_t elem)
{
    if (rows <= 0) return 0;
    const __int128 b = ((__int128)(rows - 1) * stride + n) * (__int128)elem;
    return b > ((__int128)1 << 62) ? -1 : (int64_t)b;
}

bool ranges_meet(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// The device that holds p, or a negative status.
int device_of(const void *p, const char *what)
{
    hipPointerAttribute_t a{};
    if (!p || hipPointerGetAttributes(&a, p) != hipSuccess) {
        (void)hipGetLastError();
        return api_fail(WFST_EINVAL, std::string(what) + " is not device memory");
    }
    if (a.type != hipMemoryTypeDevice && !a.isManaged)
        return api_fail(WFST_EINVAL, std::string(what) + " is not device memory");
    return a.device;
}

// Checks of one call's buffers: one that lies in an allocation already looked up in this
// call needs no second look (a lookup costs about 1 us; a caching allocator puts most of
// a call's small buffers into one block).
class Buffers {
public:
    explicit Buffers(int device) : device_(device) {}
    int check(const void *p, size_t bytes, const char *what)
    {
        const char *const at = (const char *)p;
        for (int i = 0; i < n_; ++i)
            if (p && at >= known_[i].lo && bytes <= (size_t)(known_[i].hi - known_[i].lo) && at <= known_[i].hi - bytes)
                return WFST_OK;
        Range r{nullptr, nullptr};
        const int rc = api_check_buffer(p, bytes, device_, what, &r.lo, &r.hi);
        if (rc == WFST_OK && r.lo && n_ < kMost) known_[n_++] = r;
        return rc;
    }

private:
    static constexpr int kMost = 8;
    struct Range { const char *lo, *hi; };
    int device_, n_ = 0;
    Range known_[kMost];
};

int check_stream(void *stream, int device)
{
    if (!stream) return WFST_OK;
    hipDevice_t d = -1;
    HIP_TRY(hipStreamGetDevice((hipStream_t)stream, &d));
    if (d != device) return api_fail(WFST_EINVAL, "stream belongs to another device than the operands");
    return WFST_OK;
}

int check_aligned(const void *p, size_t align, const char *what)
{
    if ((uintptr_t)p % align) return api_fail(WFST_EINVAL, std::string(what) + " is not aligned");
    return WFST_OK;
}

#define TRY(expr)                          \
    do {                                   \
        const int _rc = (expr);            \
        if (_rc < 0) return _rc;           \
    } while (0)

int check_lengths(const int32_t *lengths, int64_t rows, int32_t T, Buffers &buffers)
{
    if (!lengths) return WFST_OK;
    if (T < 1 || rows % T) return api_fail(WFST_EINVAL, "with lengths, rows must be a multiple of T >= 1");
    TRY(check_aligned(lengths, 4, "lengths"));
    return buffers.check(lengths, (size_t)(rows / T) * 4, "lengths");
}

int check_lengths(const int32_t *lengths, int64_t rows, int32_t T, int device)
{
    Buffers buffers(device);
    return check_lengths(lengths, rows, T, buffers);
}

// A range that a call writes (workspaces among them) must leave its lengths alone:
// other workgroups still read them.
int check_off_lengths(const void *p, int64_t bytes, const int32_t *lengths, int64_t rows, int32_t T, const char *what)
{
    if (!lengths || !p || !bytes || !ranges_meet(p, bytes, lengths, rows / T * 4)) return WFST_OK;
    return api_fail(WFST_EINVAL, std::string(what) + " must not overlap lengths");
}

int check_workspace(const void *w, int64_t bytes, size_t need, Buffers &buffers, const void *x, int64_t xb,
                    const void *out, int64_t ob)
{
    if (!need) return WFST_OK;
    if (!w || bytes < 0 || (size_t)bytes < need)
        return api_fail(WFST_EINVAL, "workspace must hold " + std::to_string(need) + " bytes");
    TRY(check_aligned(w, 16, "workspace"));
    TRY(buffers.check(w, need, "workspace"));
    if (ranges_meet(w, (int64_t)need, out, ob) || ranges_meet(w, (int64_t)need, x, xb))
        return api_fail(WFST_EINVAL, "workspace must not overlap the input or the output");
    return WFST_OK;
}

int check_workspace(const void *w, int64_t bytes, size_t need, int device, const void *x, int64_t xb, const void *out,
                    int64_t ob)
{
    Buffers buffers(device);
    return check_workspace(w, bytes, need, buffers, x, xb, out, ob);
}

}  // namespace

extern "C" int wfst_layer_create(const wfst_layer_desc *d, int device, void *stream, wfst_layer_t *out)
{
    return guarded([&]() -> int {
        if (!d || !out) return api_fail(WFST_EINVAL, "a pointer is null");
        *out = nullptr;
        if (d->in_features < 1 || d->in_features > (1 << 24))
            return api_fail(WFST_EINVAL, "in_features must lie in [1, 2^24]");
        if (d->out_features < 1 || d->out_features > (1 << 24))
            return api_fail(WFST_EINVAL, "out_features must lie in [1, 2^24]");
        if (d->group_size < 32 || d->group_size % 32 || d->group_size > (1 << 24))
            return api_fail(WFST_EINVAL, "group_size must be a multiple of 32 in [32, 2^24]");
        if (!dtype_ok(d->scale_dtype)) return api_fail(WFST_EINVAL, "scale_dtype is not an element type");
        if (!d->weights || !d->scales) return api_fail(WFST_EINVAL, "a pointer is null");
        int ndev = 0;
        if (hipGetDeviceCount(&ndev) != hipSuccess) ndev = 0;
        if (device < 0 || device >= ndev) return api_fail(WFST_EINVAL, "no such device");
        DeviceScope scope;
        HIP_TRY(scope.enter(device));
        const int64_t K = d->in_features, N = d->out_features;
        const int64_t ng = (K + d->group_size - 1) / d->group_size;
        const size_t ss = dtype_size(d->scale_dtype);
        TRY(check_aligned(d->scales, ss, "scales"));
        TRY(api_check_buffer(d->weights, (size_t)(N * ((K + 1) / 2)), device, "weights"));
        TRY(api_check_buffer(d->scales, (size_t)(N * ng) * ss, device, "scales"));
        if (d->zeros) TRY(api_check_buffer(d->zeros, (size_t)(N * ng), device, "zeros"));
        if (d->bias) {
            TRY(check_aligned(d->bias, 4, "bias"));
            TRY(api_check_buffer(d->bias, (size_t)N * 4, device, "bias"));
        }
        TRY(check_stream(stream, device));

        Layer l{};
        l.K = (int32_t)K;
        l.N = (int32_t)N;
        l.group = d->group_size;
        l.gpt = l.group % 128 == 0 ? 1 : (l.group == 64 ? 2 : 4);
        l.kb = (int32_t)((K + kTileK - 1) / kTileK);
        l.nt = (int32_t)((N + kTileN - 1) / kTileN);
        l.scale_dtype = d->scale_dtype;
        const auto up = [](size_t b) { return (b + 255) / 256 * 256; };
        const size_t wb = (size_t)l.nt * l.kb * 1024;
        const size_t entries = (size_t)l.nt * l.kb * kTileN * l.gpt;
        const size_t sb = up(entries * ss), zb = d->zeros ? up(entries) : 0, bb = d->bias ? up((size_t)N * 4) : 0;
        wfst_layer_s *h = new wfst_layer_s;
        hipError_t e = hipMalloc(&h->block, wb + sb + zb + bb);
        if (e != hipSuccess) {
            delete h;
            return hip_fail(e, "hipMalloc");
        }
        char *p = (char *)h->block;
        uint4 *w = (uint4 *)p;
        void *scales = p + wb;
        uint8_t *zeros = zb ? (uint8_t *)(p + wb + sb) : nullptr;
        float *bias = bb ? (float *)(p + wb + sb + zb) : nullptr;
        l.w = w;
        l.scales = scales;
        l.zeros = zeros;
        l.bias = bias;
        h->device = device;
        h->l = l;
        const LayerSource src{(const uint8_t *)d->weights, d->scales, (const uint8_t *)d->zeros,
                              (const float *)d->bias};
        e = launch_layer_pack(l, src, w, scales, zeros, bias, (hipStream_t)stream);
        if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)stream);
        if (e != hipSuccess) {
            (void)hipFree(h->block);
            delete h;
            return hip_fail(e, "wfst_layer_create");
        }
        *out = h;
        return WFST_OK;
    });
}

extern "C" int wfst_layer_release(wfst_layer_t layer)
{
    return guarded([&]() -> int {
        if (!layer) return WFST_OK;
        DeviceScope scope;
        HIP_TRY(scope.enter(layer->device));
        const hipError_t e = hipFree(layer->block);
        delete layer;
        if (e != hipSuccess) return hip_fail(e, "hipFree");
        return WFST_OK;
    });
}

extern "C" int wfst_layer_workspace(wfst_layer_t layer, int32_t x_dtype, int32_t rows, int64_t *bytes)
{
    return guarded([&]() -> int {
        if (!layer || !bytes) return api_fail(WFST_EINVAL, "a pointer is null");
        if (!dtype_ok(x_dtype)) return api_fail(WFST_EINVAL, "not an element type");
        if (rows < 0 || rows > (1 << 20) - 16) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^20 - 16]");
        *bytes = (int64_t)layer_workspace(layer->l, rows, x_dtype);
        return WFST_OK;
    });
}

namespace {

// Where the adapters' products lie in a call's workspace, behind the layer's own.
size_t adapt_offset(const Layer &l, int32_t rows, int32_t x_dtype)
{
    return (layer_workspace(l, rows, x_dtype) + 255) / 256 * 256;
}

size_t adapt_workspace(const Layer &l, const Adapters &a, int32_t rows, int32_t x_dtype)
{
    const AdaptBytes b = adapt_bytes(a, rows);
    return adapt_offset(l, rows, x_dtype) + b.h + b.lists + b.counts;
}

int check_same_layer(const Layer &l, int device, wfst_adapters_t ad)
{
    if (ad->a.K != l.K || ad->a.N != l.N) return api_fail(WFST_EINVAL, "the adapters are of a layer of another size");
    if (ad->device != device) return api_fail(WFST_EINVAL, "the adapters are on another device than the layer");
    return WFST_OK;
}

// The layer's logits, with adapters where ad is given.
int layer_logits(wfst_layer_t layer, wfst_adapters_t ad, const int32_t *ids, int32_t rows_per_id, const void *x,
                 int32_t x_dtype, int64_t x_stride, int32_t rows, const int32_t *lengths, int32_t T, void *out,
                 int32_t out_dtype, int64_t out_stride, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!layer) return api_fail(WFST_EINVAL, "layer is null");
    const Layer &l = layer->l;
    if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return api_fail(WFST_EINVAL, "not an element type");
    if (rows < 0 || rows > (1 << 20) - 16) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^20 - 16]");
    if (ad) TRY(check_same_layer(l, layer->device, ad));
    if (rows == 0) return WFST_OK;
    if (!x || !out || (ad && !ids)) return api_fail(WFST_EINVAL, "a pointer is null");
    if (ad && (rows_per_id < 1 || rows % rows_per_id))
        return api_fail(WFST_EINVAL, "rows must be a multiple of rows_per_id >= 1");
    if (rows > 1 && (x_stride < l.K || out_stride < l.N))
        return api_fail(WFST_EINVAL, "a row stride is smaller than its row");
    const size_t xe = dtype_size(x_dtype), oe = dtype_size(out_dtype);
    const int64_t xb = span_bytes(rows, l.K, x_stride, xe), ob = span_bytes(rows, l.N, out_stride, oe);
    if (xb < 0 || ob < 0) return api_fail(WFST_EINVAL, "a tensor is too large");
    DeviceScope scope;
    HIP_TRY(scope.enter(layer->device));
    TRY(check_aligned(x, xe, "x"));
    TRY(check_aligned(out, oe, "out"));
    Buffers buffers(layer->device);
    TRY(buffers.check(x, (size_t)xb, "x"));
    TRY(buffers.check(out, (size_t)ob, "out"));
    TRY(check_lengths(lengths, rows, T, buffers));
    TRY(check_stream(stream, layer->device));
    if (ranges_meet(x, xb, out, ob)) return api_fail(WFST_EINVAL, "out must not overlap x");
    const size_t need = ad ? adapt_workspace(l, ad->a, rows, x_dtype) : layer_workspace(l, rows, x_dtype);
    TRY(check_workspace(workspace, workspace_bytes, need, buffers, x, xb, out, ob));
    TRY(check_off_lengths(out, ob, lengths, rows, T, "out"));
    TRY(check_off_lengths(workspace, (int64_t)need, lengths, rows, T, "workspace"));
    LayerCall c{x, out, x_stride, out_stride, rows, x_dtype, out_dtype, {lengths, T}, workspace, {}};
    if (ad) {
        const int64_t ib = (int64_t)(rows / rows_per_id) * 4;
        TRY(check_aligned(ids, 4, "ids"));
        TRY(buffers.check(ids, (size_t)ib, "ids"));
        if (ranges_meet(ids, ib, out, ob) || ranges_meet(ids, ib, workspace, (int64_t)need))
            return api_fail(WFST_EINVAL, "out and workspace must not overlap ids");
        char *h = (char *)workspace + adapt_offset(l, rows, x_dtype);
        const AdaptBytes b = adapt_bytes(ad->a, rows);
        c.ad = {ad->a, ids, rows_per_id, h, (uint4 *)(h + b.h), (int32_t *)(h + b.h + b.lists), 0, 0};
    }
    HIP_TRY(launch_layer(l, c, (hipStream_t)stream));
    return WFST_OK;
}

}  // namespace

extern "C" int wfst_layer_logits(wfst_layer_t layer, const void *x, int32_t x_dtype, int64_t x_stride, int32_t rows,
                                 const int32_t *lengths, int32_t T, void *out, int32_t out_dtype, int64_t out_stride,
                                 void *workspace, int64_t workspace_bytes, void *stream)
{
    return guarded([&]() -> int {
        return layer_logits(layer, nullptr, nullptr, 1, x, x_dtype, x_stride, rows, lengths, T, out, out_dtype,
                            out_stride, workspace, workspace_bytes, stream);
    });
}

extern "C" int wfst_layer_adapted_logits(wfst_layer_t layer, wfst_adapters_t adapters, const int32_t *ids,
                                         int32_t rows_per_id, const void *x, int32_t x_dtype, int64_t x_stride,
                                         int32_t rows, const int32_t *lengths, int32_t T, void *out, int32_t out_dtype,
                                         int64_t out_stride, void *workspace, int64_t workspace_bytes, void *stream)
{
    return guarded([&]() -> int {
        if (!adapters) return api_fail(WFST_EINVAL, "adapters is null");
        return layer_logits(layer, adapters, ids, rows_per_id, x, x_dtype, x_stride, rows, lengths, T, out, out_dtype,
                            out_stride, workspace, workspace_bytes, stream);
    });
}

extern "C" int wfst_layer_adapted_workspace(wfst_layer_t layer, wfst_adapters_t adapters, int32_t x_dtype,
                                            int32_t rows, int64_t *bytes)
{
    return guarded([&]() -> int {
        if (!layer || !adapters || !bytes) return api_fail(WFST_EINVAL, "a pointer is null");
        if (!dtype_ok(x_dtype)) return api_fail(WFST_EINVAL, "not an element type");
        if (rows < 0 || rows > (1 << 20) - 16) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^20 - 16]");
        TRY(check_same_layer(layer->l, layer->device, adapters));
        *bytes = (int64_t)adapt_workspace(layer->l, adapters->a, rows, x_dtype);
        return WFST_OK;
    });
}

extern "C" int wfst_adapters_create(const wfst_adapters_desc *d, int device, void *stream, wfst_adapters_t *out)
{
    return guarded([&]() -> int {
        if (!d || !out) return api_fail(WFST_EINVAL, "a pointer is null");
        *out = nullptr;
        if (d->in_features < 1 || d->in_features > (1 << 24))
            return api_fail(WFST_EINVAL, "in_features must lie in [1, 2^24]");
        if (d->out_features < 1 || d->out_features > (1 << 24))
            return api_fail(WFST_EINVAL, "out_features must lie in [1, 2^24]");
        if (d->slots < 1 || d->slots > (1 << 16)) return api_fail(WFST_EINVAL, "slots must lie in [1, 2^16]");
        if (d->rank < 1 || d->rank > 128) return api_fail(WFST_EINVAL, "rank must lie in [1, 128]");
        if (!dtype_ok(d->dtype)) return api_fail(WFST_EINVAL, "dtype is not an element type");
        int ndev = 0;
        if (hipGetDeviceCount(&ndev) != hipSuccess) ndev = 0;
        if (device < 0 || device >= ndev) return api_fail(WFST_EINVAL, "no such device");
        DeviceScope scope;
        HIP_TRY(scope.enter(device));
        TRY(check_stream(stream, device));
        Adapters a{};
        a.K = d->in_features;
        a.N = d->out_features;
        a.slots = d->slots;
        a.rank = d->rank;
        a.rb = (d->rank + 15) / 16;
        a.kp = (d->in_features + 31) / 32 * 32;
        a.nt = (d->out_features + kTileN - 1) / kTileN;
        a.dtype = d->dtype;
        const auto up = [](size_t b) { return (b + 255) / 256 * 256; };
        const size_t es = dtype_size(a.dtype), n = (size_t)a.slots * a.rb * 16;
        const size_t db = up(n * a.kp * es), ub = up(n * a.nt * kTileN * es), sb = up((size_t)a.slots * 4);
        wfst_adapters_s *h = new wfst_adapters_s;
        hipError_t e = hipMalloc(&h->block, db + ub + 2 * sb);
        if (e != hipSuccess) {
            delete h;
            return hip_fail(e, "hipMalloc");
        }
        char *p = (char *)h->block;
        a.down = p;
        a.up = p + db;
        a.scales = (float *)(p + db + ub);
        a.ranks = (int32_t *)(p + db + ub + sb);
        h->device = device;
        h->a = a;
        e = launch_adapters_clear(a, (hipStream_t)stream);
        if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)stream);
        if (e != hipSuccess) {
            (void)hipFree(h->block);
            delete h;
            return hip_fail(e, "wfst_adapters_create");
        }
        *out = h;
        return WFST_OK;
    });
}

extern "C" int wfst_adapters_release(wfst_adapters_t adapters)
{
    return guarded([&]() -> int {
        if (!adapters) return WFST_OK;
        DeviceScope scope;
        HIP_TRY(scope.enter(adapters->device));
        const hipError_t e = hipFree(adapters->block);
        delete adapters;
        if (e != hipSuccess) return hip_fail(e, "hipFree");
        return WFST_OK;
    });
}

extern "C" int wfst_adapters_load(wfst_adapters_t adapters, int32_t slot, int32_t rank, const void *down,
                                  int64_t down_stride, const void *up, int64_t up_stride, float scale, void *stream)
{
    return guarded([&]() -> int {
        if (!adapters) return api_fail(WFST_EINVAL, "adapters is null");
        const Adapters &a = adapters->a;
        if (slot < 0 || slot >= a.slots) return api_fail(WFST_EINVAL, "slot must lie in [0, slots)");
        if (rank < 0 || rank > a.rank) return api_fail(WFST_EINVAL, "rank must lie in [0, the adapters' rank]");
        if (!std::isfinite(scale)) return api_fail(WFST_EINVAL, "scale must be finite");
        if (rank && (!down || !up)) return api_fail(WFST_EINVAL, "a pointer is null");
        if ((rank > 1 && down_stride < a.K) || (rank && a.N > 1 && up_stride < rank))
            return api_fail(WFST_EINVAL, "a row stride is smaller than its row");
        const size_t es = dtype_size(a.dtype);
        const int64_t db = span_bytes(rank, a.K, down_stride, es), ub = span_bytes(rank ? a.N : 0, rank, up_stride, es);
        if (db < 0 || ub < 0) return api_fail(WFST_EINVAL, "a tensor is too large");
        DeviceScope scope;
        HIP_TRY(scope.enter(adapters->device));
        if (rank) {
            TRY(check_aligned(down, es, "down"));
            TRY(check_aligned(up, es, "up"));
            TRY(api_check_buffer(down, (size_t)db, adapters->device, "down"));
            TRY(api_check_buffer(up, (size_t)ub, adapters->device, "up"));
        }
        TRY(check_stream(stream, adapters->device));
        HIP_TRY(launch_adapter_load(a, slot, {down, up, down_stride, up_stride, rank, scale}, (hipStream_t)stream));
        return WFST_OK;
    });
}

extern "C" int wfst_log_softmax(const void *x, int32_t x_dtype, int64_t x_stride, int64_t rows, int32_t V, float scale,
                                const float *bias, const int32_t *lengths, int32_t T, void *out, int32_t out_dtype,
                                int64_t out_stride, void *workspace, int64_t workspace_bytes, void *stream)
{
    return guarded([&]() -> int {
        if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return api_fail(WFST_EINVAL, "not an element type");
        if (rows < 0 || rows > ((int64_t)1 << 40)) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^40]");
        if (V < 1 || V > (1 << 24)) return api_fail(WFST_EINVAL, "V must lie in [1, 2^24]");
        if (!std::isfinite(scale)) return api_fail(WFST_EINVAL, "scale must be finite");
        if (rows == 0) return WFST_OK;
        if (!x || !out) return api_fail(WFST_EINVAL, "a pointer is null");
        if (rows > 1 && (x_stride < V || out_stride < V))
            return api_fail(WFST_EINVAL, "a row stride is smaller than its row");
        const size_t xe = dtype_size(x_dtype), oe = dtype_size(out_dtype);
        const int64_t xb = span_bytes(rows, V, x_stride, xe), ob = span_bytes(rows, V, out_stride, oe);
        if (xb < 0 || ob < 0) return api_fail(WFST_EINVAL, "a tensor is too large");
        const int device = device_of(x, "x");
        if (device < 0) return device;
        DeviceScope scope;
        HIP_TRY(scope.enter(device));
        TRY(check_aligned(x, xe, "x"));
        TRY(check_aligned(out, oe, "out"));
        TRY(api_check_buffer(x, (size_t)xb, device, "x"));
        TRY(api_check_buffer(out, (size_t)ob, device, "out"));
        if (bias) {
            TRY(check_aligned(bias, 4, "bias"));
            TRY(api_check_buffer(bias, (size_t)V * 4, device, "bias"));
        }
        TRY(check_lengths(lengths, rows, T, device));
        TRY(check_stream(stream, device));
        const bool in_place = x == out && x_dtype == out_dtype && (rows == 1 || x_stride == out_stride);
        if (!in_place && ranges_meet(x, xb, out, ob))
            return api_fail(WFST_EINVAL, "out must be x itself (same type and stride) or not overlap it");
        if (bias && ranges_meet(bias, (int64_t)V * 4, out, ob))
            return api_fail(WFST_EINVAL, "out must not overlap bias");
        const size_t need = norm_workspace(rows, V, x_dtype, out_dtype);
        TRY(check_workspace(workspace, workspace_bytes, need, device, x, xb, out, ob));
        if (need && bias && ranges_meet(workspace, (int64_t)need, bias, (int64_t)V * 4))
            return api_fail(WFST_EINVAL, "workspace must not overlap bias");
        TRY(check_off_lengths(out, ob, lengths, rows, T, "out"));
        TRY(check_off_lengths(workspace, (int64_t)need, lengths, rows, T, "workspace"));
        const NormCall c{x, out, bias, x_stride, out_stride, rows, V, x_dtype, out_dtype, scale, {lengths, T}, workspace};
        HIP_TRY(launch_log_softmax(c, (hipStream_t)stream));
        return WFST_OK;
    });
}

extern "C" int wfst_log_softmax_workspace(int32_t x_dtype, int64_t rows, int32_t V, int32_t out_dtype, int64_t *bytes)
{
    return guarded([&]() -> int {
        if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return api_fail(WFST_EINVAL, "not an element type");
        if (rows < 0 || rows > ((int64_t)1 << 40)) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^40]");
        if (V < 1 || V > (1 << 24)) return api_fail(WFST_EINVAL, "V must lie in [1, 2^24]");
        if (!bytes) return api_fail(WFST_EINVAL, "a pointer is null");
        *bytes = (int64_t)norm_workspace(rows, V, x_dtype, out_dtype);
        return WFST_OK;
    });
}

extern "C" int wfst_sample_workspace(int32_t x_dtype, int64_t rows, int32_t V, int64_t *bytes)
{
    return guarded([&]() -> int {
        if (!dtype_ok(x_dtype)) return api_fail(WFST_EINVAL, "not an element type");
        if (rows < 0 || rows > ((int64_t)1 << 40)) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^40]");
        if (V < 1 || V > (1 << 24)) return api_fail(WFST_EINVAL, "V must lie in [1, 2^24]");
        if (!bytes) return api_fail(WFST_EINVAL, "a pointer is null");
        *bytes = (int64_t)sample_workspace(rows, V, x_dtype);
        return WFST_OK;
    });
}

extern "C" int wfst_sample(const void *x, int32_t x_dtype, int64_t x_stride, int64_t rows, int32_t V, const float *u,
                           const wfst_sample_config *cfg, const int32_t *lengths, int32_t T, int32_t *out_tokens,
                           float *out_log_probs, int32_t *out_kept, void *workspace, int64_t workspace_bytes,
                           void *stream)
{
    return guarded([&]() -> int {
        if (!cfg) return api_fail(WFST_EINVAL, "config is null");
        if (!dtype_ok(x_dtype)) return api_fail(WFST_EINVAL, "not an element type");
        if (rows < 0 || rows > ((int64_t)1 << 40)) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^40]");
        if (V < 1 || V > (1 << 24)) return api_fail(WFST_EINVAL, "V must lie in [1, 2^24]");
        if (!cfg->temperatures && !(cfg->temperature >= 0.0f && std::isfinite(cfg->temperature)))
            return api_fail(WFST_EINVAL, "temperature must be finite and not negative");
        if (!cfg->top_ks && cfg->top_k < 0) return api_fail(WFST_EINVAL, "top_k must not be negative");
        if (!cfg->top_ps && !(cfg->top_p >= 0.0f && cfg->top_p <= 1.0f))
            return api_fail(WFST_EINVAL, "top_p must lie in [0, 1]");
        if (!cfg->min_ps && !(cfg->min_p >= 0.0f && cfg->min_p <= 1.0f))
            return api_fail(WFST_EINVAL, "min_p must lie in [0, 1]");
        if (rows == 0) return WFST_OK;
        if (!x || !u || !out_tokens) return api_fail(WFST_EINVAL, "a pointer is null");
        if (rows > 1 && x_stride < V) return api_fail(WFST_EINVAL, "a row stride is smaller than its row");
        const size_t xe = dtype_size(x_dtype);
        const int64_t xb = span_bytes(rows, V, x_stride, xe), rb = span_bytes(rows, 1, 1, 4);
        if (xb < 0 || rb < 0) return api_fail(WFST_EINVAL, "a tensor is too large");
        const int device = device_of(x, "scores");
        if (device < 0) return device;
        DeviceScope scope;
        HIP_TRY(scope.enter(device));
        TRY(check_aligned(x, xe, "scores"));
        TRY(api_check_buffer(x, (size_t)xb, device, "scores"));
        const struct { const void *p; const char *name; bool out; } row_args[] = {
            {u, "u", false}, {cfg->temperatures, "temperatures", false}, {cfg->top_ks, "top_ks", false},
            {cfg->top_ps, "top_ps", false}, {cfg->min_ps, "min_ps", false}, {out_tokens, "out_tokens", true},
            {out_log_probs, "out_log_probs", true}, {out_kept, "out_kept", true}};
        for (const auto &a : row_args) {
            if (!a.p) continue;
            TRY(check_aligned(a.p, 4, a.name));
            TRY(api_check_buffer(a.p, (size_t)rb, device, a.name));
        }
        for (const auto &o : row_args) {
            if (!o.out || !o.p) continue;
            if (ranges_meet(o.p, rb, x, xb)) return api_fail(WFST_EINVAL, "an output overlaps the scores");
            for (const auto &a : row_args)
                if (a.p && &a != &o && ranges_meet(o.p, rb, a.p, rb))
                    return api_fail(WFST_EINVAL, std::string(o.name) + " overlaps " + a.name);
        }
        TRY(check_lengths(lengths, rows, T, device));
        TRY(check_stream(stream, device));
        const size_t need = sample_workspace(rows, V, x_dtype);
        TRY(check_workspace(workspace, workspace_bytes, need, device, x, xb, out_tokens, rb));
        if (need)
            for (const auto &a : row_args)
                if (a.p && ranges_meet(workspace, (int64_t)need, a.p, rb))
                    return api_fail(WFST_EINVAL, std::string("workspace overlaps ") + a.name);
        for (const auto &o : row_args)
            if (o.out) TRY(check_off_lengths(o.p, rb, lengths, rows, T, o.name));
        TRY(check_off_lengths(workspace, (int64_t)need, lengths, rows, T, "workspace"));
        SampleCall c{};
        c.x = x;
        c.x_stride = x_stride;
        c.rows = rows;
        c.V = V;
        c.x_dtype = x_dtype;
        c.u = u;
        c.temperature = cfg->temperature;
        c.top_k = cfg->top_k;
        c.top_p = cfg->top_p;
        c.min_p = cfg->min_p;
        c.temperatures = (const float *)cfg->temperatures;
        c.top_ks = (const int32_t *)cfg->top_ks;
        c.top_ps = (const float *)cfg->top_ps;
        c.min_ps = (const float *)cfg->min_ps;
        c.token = out_tokens;
        c.log_prob = out_log_probs;
        c.kept = out_kept;
        c.set = {lengths, T};
        c.workspace = workspace;
        HIP_TRY(launch_sample(c, (hipStream_t)stream));
        return WFST_OK;
    });
}

namespace {

int check_token_sizes(int32_t x_dtype, int64_t rows, int32_t V, int32_t C, int32_t top_n)
{
    if (!dtype_ok(x_dtype)) return api_fail(WFST_EINVAL, "not an element type");
    if (rows < 0 || rows > ((int64_t)1 << 40)) return api_fail(WFST_EINVAL, "rows must lie in [0, 2^40]");
    if (V < 1 || V > (1 << 24)) return api_fail(WFST_EINVAL, "V must lie in [1, 2^24]");
    if (C < 0 || C > kMaxTokens) return api_fail(WFST_EINVAL, "tokens_per_row must lie in [0, 256]");
    if (top_n < 0 || top_n > kMaxTop) return api_fail(WFST_EINVAL, "top_n must lie in [0, 64]");
    return WFST_OK;
}

}  // namespace

extern "C" int wfst_token_scores_workspace(int32_t x_dtype, int64_t rows, int32_t V, int32_t tokens_per_row,
                                           int32_t top_n, int64_t *bytes)
{
    return guarded([&]() -> int {
        TRY(check_token_sizes(x_dtype, rows, V, tokens_per_row, top_n));
        if (!bytes) return api_fail(WFST_EINVAL, "a pointer is null");
        *bytes = (int64_t)token_workspace(rows, V, tokens_per_row, top_n, x_dtype);
        return WFST_OK;
    });
}

extern "C" int wfst_token_scores(const void *x, int32_t x_dtype, int64_t x_stride, int64_t rows, int32_t V,
                                 const int32_t *tokens, int32_t tokens_per_row, int32_t top_n, float temperature,
                                 const float *temperatures, const int32_t *lengths, int32_t T,
                                 const wfst_token_scores_out *out, void *workspace, int64_t workspace_bytes,
                                 void *stream)
{
    return guarded([&]() -> int {
        const int32_t C = tokens_per_row;
        if (!out) return api_fail(WFST_EINVAL, "out is null");
        TRY(check_token_sizes(x_dtype, rows, V, C, top_n));
        if (!temperatures && !(temperature >= 0.0f && std::isfinite(temperature)))
            return api_fail(WFST_EINVAL, "temperature must be finite and not negative");
        if (rows == 0) return WFST_OK;
        if (!x || (C && (!tokens || !out->log_probs || !out->ranks)) ||
            (top_n && (!out->top_tokens || !out->top_log_probs)))
            return api_fail(WFST_EINVAL, "a pointer is null");
        if (rows > 1 && x_stride < V) return api_fail(WFST_EINVAL, "a row stride is smaller than its row");
        const size_t xe = dtype_size(x_dtype);
        const int64_t xb = span_bytes(rows, V, x_stride, xe);
        if (xb < 0) return api_fail(WFST_EINVAL, "a tensor is too large");
        const int device = device_of(x, "scores");
        if (device < 0) return device;
        DeviceScope scope;
        HIP_TRY(scope.enter(device));
        TRY(check_aligned(x, xe, "scores"));
        Buffers buffers(device);
        TRY(buffers.check(x, (size_t)xb, "scores"));
        const int64_t cb = rows * C * 4, nb = rows * top_n * 4;
        const struct { const void *p; int64_t bytes; const char *name; bool out; } args[] = {
            {C ? tokens : nullptr, cb, "tokens", false}, {temperatures, rows * 4, "temperatures", false},
            {C ? out->log_probs : nullptr, cb, "log_probs", true}, {C ? out->ranks : nullptr, cb, "ranks", true},
            {out->entropies, rows * 4, "entropies", true},
            {top_n ? out->top_tokens : nullptr, nb, "top_tokens", true},
            {top_n ? out->top_log_probs : nullptr, nb, "top_log_probs", true}};
        bool any = false;
        for (const auto &a : args) {
            if (!a.p) continue;
            any |= a.out;
            TRY(check_aligned(a.p, 4, a.name));
            TRY(buffers.check(a.p, (size_t)a.bytes, a.name));
        }
        if (!any) return api_fail(WFST_EINVAL, "no output is wanted");
        for (const auto &o : args) {
            if (!o.out || !o.p) continue;
            if (ranges_meet(o.p, o.bytes, x, xb)) return api_fail(WFST_EINVAL, "an output overlaps the scores");
            for (const auto &a : args)
                if (a.p && &a != &o && ranges_meet(o.p, o.bytes, a.p, a.bytes))
                    return api_fail(WFST_EINVAL, std::string(o.name) + " overlaps " + a.name);
        }
        TRY(check_lengths(lengths, rows, T, buffers));
        TRY(check_stream(stream, device));
        const size_t need = token_workspace(rows, V, C, top_n, x_dtype);
        TRY(check_workspace(workspace, workspace_bytes, need, buffers, x, xb, nullptr, 0));
        for (const auto &a : args) {
            if (need && a.p && ranges_meet(workspace, (int64_t)need, a.p, a.bytes))
                return api_fail(WFST_EINVAL, std::string("workspace overlaps ") + a.name);
            if (a.out) TRY(check_off_lengths(a.p, a.bytes, lengths, rows, T, a.name));
        }
        TRY(check_off_lengths(workspace, (int64_t)need, lengths, rows, T, "workspace"));
        TokenCall c{};
        c.x = x;
        c.x_stride = x_stride;
        c.rows = rows;
        c.V = V;
        c.x_dtype = x_dtype;
        c.tokens = tokens;
        c.C = C;
        c.top_n = top_n;
        c.temperature = temperature;
        c.temperatures = temperatures;
        c.log_probs = (float *)out->log_probs;
        c.ranks = (int32_t *)out->ranks;
        c.entropies = (float *)out->entropies;
        c.top_tokens = (int32_t *)out->top_tokens;
        c.top_log_probs = (float *)out->top_log_probs;
        c.set = {lengths, T};
        c.workspace = workspace;
        HIP_TRY(launch_token_scores(c, (hipStream_t)stream));
        return WFST_OK;
    });
}
