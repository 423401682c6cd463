// delta_api.cu -- the C entry points of the gated delta rule and of gradient clipping (declared in
// include/ttt.h): argument validation, nothing computed here.
#include <algorithm>
#include <cmath>
#include <new>

#include "delta.cuh"

namespace ttt {
size_t clip_ws_bytes(int n);
ttt_status launch_clip(const void* const* in, void* const* out, const long long* counts, const int* dtypes, int n, float max_norm,
                       float* norm_out, void* ws, cudaStream_t st);

namespace gd {

// Whether p is memory of the current device `dev`, or managed.
static bool device_ptr(const void* p, int dev) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();   // clear the non-sticky error
        return false;
    }
    return (a.type == cudaMemoryTypeDevice && a.device == dev) || a.type == cudaMemoryTypeManaged;
}
static int current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
    return dev;
}
static bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

static ttt_status check_delta_shape(const ttt_delta_shape* s) {
    if (!s) return TTT_ERR_INVALID_ARG;
    if (s->batch < 1 || s->qk_heads < 1 || s->heads < 1 || s->tokens < 1 || s->d_k < 1 || s->d_v < 1) return TTT_ERR_INVALID_ARG;
    if (s->heads % s->qk_heads) return TTT_ERR_INVALID_ARG;
    if (s->dtype != TTT_FP32 && s->dtype != TTT_BF16) return TTT_ERR_INVALID_ARG;
    if (s->tokens > (1 << 30) || (long long)s->batch * s->heads > (1LL << 24)) return TTT_ERR_INVALID_ARG;
    if ((s->d_k != 64 && s->d_k != 128) || (s->d_v != 64 && s->d_v != 128)) return TTT_ERR_UNSUPPORTED;
    // one warp per (image, head, chunk of 32 tokens) in a grid of at most 2^31 - 1 CTAs
    if ((long long)s->batch * s->heads * ((s->tokens + CT - 1LL) / CT) > (1LL << 31) - 1) return TTT_ERR_UNSUPPORTED;
    return TTT_OK;
}

static Dims dims_of(const ttt_delta_shape& s) {
    Dims d{};
    d.B = s.batch; d.hk = s.qk_heads; d.h = s.heads; d.r = s.heads / s.qk_heads;
    d.N = s.tokens; d.dk = s.d_k; d.dv = s.d_v;
    d.nc = (d.N + CT - 1) / CT;
    d.gt = group_tokens(s.dtype == TTT_FP32);
    d.ng = (d.N + d.gt - 1) / d.gt;
    return d;
}

// One tensor of a call as the checks see it: extents and strides in elements of `esz` bytes.
struct Slab {
    const char* p;
    long long n[3], st[3];        // batch, heads, tokens
    int width, esz;
    long long image() const { return ((n[1] - 1) * st[1] + (n[2] - 1) * st[2] + width) * esz; }   // bytes from the first to past the last
    long long span() const { return image() + (n[0] - 1) * st[0] * esz; }
};

// Whether two elements of the slab may share an address: its dimensions, ordered by stride, have to nest.
static bool self_overlaps(const Slab& s) {
    int o[3] = {0, 1, 2};
    std::sort(o, o + 3, [&](int a, int b) { return s.st[a] < s.st[b]; });
    long long e = s.width;
    for (int i : o) {
        if (s.n[i] == 1) continue;
        if (s.st[i] < e) return true;
        e += (s.n[i] - 1) * s.st[i];
    }
    return false;
}

// Whether two slabs may share memory.  Slabs whose address ranges meet are still apart if they interleave: cut
// from the rows of one larger buffer (the same token stride), at ranges of a row that do not meet.
static bool may_overlap(const Slab& a, const Slab& b) {
    if (!(a.p < b.p + b.span() && b.p < a.p + a.span())) return false;
    if (a.esz != b.esz) return true;
    long long row = 0;
    for (const Slab* s : {&a, &b})
        if (s->n[2] > 1) {
            const long long r = s->st[2] * s->esz;
            if (row != 0 && row != r) return true;
            row = r;
        }
    if (row == 0) return true;
    // equal batch strides that keep the images apart: image b of one can only meet image b of the other
    const long long apart = (b.p > a.p ? b.p - a.p : a.p - b.p) + std::max(a.image(), b.image());
    const bool by_image = a.n[0] == b.n[0] && a.st[0] == b.st[0] && apart <= a.st[0] * a.esz;
    long long lo[2], hi[2];
    const Slab* s[2] = {&a, &b};
    for (int i = 0; i < 2; ++i) {
        const bool whole_rows = s[i]->n[0] == 1 || (s[i]->st[0] * s[i]->esz) % row == 0;
        if (!whole_rows && !by_image) return true;
        const long long w = ((s[i]->n[1] - 1) * s[i]->st[1] + s[i]->width) * s[i]->esz;
        if (w > row) return true;
        lo[i] = i == 0 ? 0 : ((b.p - a.p) % row + row) % row;
        hi[i] = lo[i] + w;
    }
    // a's columns are [0, hi0); b's are [lo1, hi1), which may wrap past the row's end
    return lo[1] < hi[0] || hi[1] > row;
}

static ttt_status add_view(const ttt_view* v, int batch, int heads, int tokens, int width, int esz, View* out, Slab* slab) {
    if (!v || !v->data) return TTT_ERR_INVALID_ARG;
    if (v->batch_stride < 0 || v->head_stride < 0 || v->token_stride < 0) return TTT_ERR_INVALID_ARG;
    const size_t align = width > 1 ? 16 : esz;
    if (misaligned(v->data, align)) return TTT_ERR_ALIGNMENT;
    Slab s{static_cast<const char*>(v->data), {batch, heads, tokens}, {v->batch_stride, v->head_stride, v->token_stride}, width, esz};
    for (int i = 0; i < 3; ++i) {
        if (s.n[i] == 1) s.st[i] = 0;
        else if (width > 1 && (s.st[i] * esz) % 16) return TTT_ERR_ALIGNMENT;
    }
    *out = View{static_cast<char*>(v->data), s.st[0], s.st[1], s.st[2]};
    *slab = s;
    return TTT_OK;
}

// The views of a call: inputs may overlap one another and be broadcast (stride 0), outputs may overlap nothing.
struct Arguments {
    const ttt_delta_shape* s;
    Slab slabs[16];               // a backward call's 11 views, W0, dW1, dW0, workspace and lengths
    bool output[16];
    int n = 0;
    ttt_status st = TTT_OK;

    void tokens(const ttt_view* v, int heads, int width, View* out, bool is_output, bool fp32 = false) {
        if (st != TTT_OK) return;
        st = add_view(v, s->batch, heads, s->tokens, width, fp32 || s->dtype == TTT_FP32 ? 4 : 2, out, &slabs[n]);
        output[n++] = is_output;
    }
    void flat(const void* p, long long bytes, bool is_output, size_t align = 16) {
        if (st != TTT_OK || !p) return;
        if (misaligned(p, align)) { st = TTT_ERR_ALIGNMENT; return; }
        slabs[n] = Slab{static_cast<const char*>(p), {1, 1, 1}, {0, 0, 0}, 1, 1};
        slabs[n].n[0] = bytes;              // `bytes` single bytes in a row
        slabs[n].st[0] = 1;
        output[n++] = is_output;
    }
    ttt_status finish() {
        if (st != TTT_OK) return st;
        for (int i = 0; i < n; ++i) {
            if (output[i] && self_overlaps(slabs[i])) return TTT_ERR_INVALID_ARG;
            for (int j = 0; j < i; ++j)
                if ((output[i] || output[j]) && may_overlap(slabs[i], slabs[j])) return TTT_ERR_INVALID_ARG;
        }
        const int dev = current_device();
        for (int i = 0; i < n; ++i)
            if (!device_ptr(slabs[i].p, dev)) return TTT_ERR_INVALID_ARG;
        return ttt_last_error();
    }
};

// SMs of the current device (148 if it cannot be asked; the launch then reports why).
static int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    return n;
}

}  // namespace gd
}  // namespace ttt

using namespace ttt;
using namespace ttt::gd;

extern "C" {

size_t ttt_gated_delta_workspace_bytes(int backward, const ttt_delta_shape* s) {
    if (check_delta_shape(s) != TTT_OK) return 0;
    const Dims d = dims_of(*s);
    return backward ? backward_ws_bytes(d, s->dtype == TTT_FP32) : forward_ws_bytes(d, s->dtype == TTT_FP32);
}

ttt_status ttt_forward_gated_delta(const ttt_view* Q, const ttt_view* K, const ttt_view* V, const ttt_view* G, const ttt_view* Beta,
                                   const float* W0, int w0_shared, const int* lengths, float scale, const ttt_view* Z, float* W1_out,
                                   const ttt_delta_shape* s, void* ws, size_t ws_bytes, void* stream) {
    ttt_status st = check_delta_shape(s);
    if (st != TTT_OK) return st;
    if (!std::isfinite(scale)) return TTT_ERR_INVALID_ARG;
    gd::Call c{};
    c.d = dims_of(*s);
    c.fp32 = s->dtype == TTT_FP32;
    c.d.lengths = lengths;
    c.d.scale = scale;
    const long long state = (long long)s->heads * s->d_v * s->d_k * 4, states = state * s->batch;
    Arguments k{s};
    k.tokens(Q, s->qk_heads, s->d_k, &c.Q, false);
    k.tokens(K, s->qk_heads, s->d_k, &c.K, false);
    k.tokens(V, s->heads, s->d_v, &c.V, false);
    k.tokens(G, s->heads, 1, &c.G, false, true);
    k.tokens(Beta, s->heads, 1, &c.Beta, false, true);
    k.tokens(Z, s->heads, s->d_v, &c.Z, true);
    k.flat(lengths, 4LL * s->batch, false, 4);
    k.flat(W0, w0_shared ? state : states, false);
    k.flat(W1_out, states, true);
    if (k.st != TTT_OK) return k.st;
    const size_t need = forward_ws_bytes(c.d, c.fp32);
    if (!ws || ws_bytes < need) return TTT_ERR_WORKSPACE;
    if (misaligned(ws, 256)) return TTT_ERR_ALIGNMENT;
    k.flat(ws, (long long)need, true);
    st = k.finish();
    if (st != TTT_OK) return st;
    c.W0 = W0;
    c.w0_bs = w0_shared ? 0 : state / 4;
    c.W1_out = W1_out;
    c.ws = static_cast<uint8_t*>(ws);
    c.wait_ns = wait_limit_ns();
    c.sms = sm_count();
    c.stream = static_cast<cudaStream_t>(stream);
    return launch_forward(c);
}

ttt_status ttt_backward_gated_delta(const ttt_view* Q, const ttt_view* K, const ttt_view* V, const ttt_view* G, const ttt_view* Beta,
                                    const float* W0, int w0_shared, const int* lengths, float scale, const ttt_view* dZ,
                                    const float* dW1, const ttt_delta_shape* s, void* ws, size_t ws_bytes, const ttt_view* dQ,
                                    const ttt_view* dK, const ttt_view* dV, const ttt_view* dG, const ttt_view* dBeta, float* dW0_out,
                                    void* stream) {
    ttt_status st = check_delta_shape(s);
    if (st != TTT_OK) return st;
    if (!std::isfinite(scale) || (dW0_out && !W0)) return TTT_ERR_INVALID_ARG;
    gd::Call c{};
    c.d = dims_of(*s);
    c.fp32 = s->dtype == TTT_FP32;
    c.d.lengths = lengths;
    c.d.scale = scale;
    const long long state = (long long)s->heads * s->d_v * s->d_k * 4, states = state * s->batch;
    Arguments k{s};
    k.tokens(Q, s->qk_heads, s->d_k, &c.Q, false);
    k.tokens(K, s->qk_heads, s->d_k, &c.K, false);
    k.tokens(V, s->heads, s->d_v, &c.V, false);
    k.tokens(G, s->heads, 1, &c.G, false, true);
    k.tokens(Beta, s->heads, 1, &c.Beta, false, true);
    k.tokens(dZ, s->heads, s->d_v, &c.Z, false);
    k.tokens(dQ, s->qk_heads, s->d_k, &c.dQ, true);
    k.tokens(dK, s->qk_heads, s->d_k, &c.dK, true);
    k.tokens(dV, s->heads, s->d_v, &c.dV, true);
    k.tokens(dG, s->heads, 1, &c.dG, true, true);
    k.tokens(dBeta, s->heads, 1, &c.dBeta, true, true);
    k.flat(lengths, 4LL * s->batch, false, 4);
    k.flat(W0, w0_shared ? state : states, false);
    k.flat(dW1, states, false);
    k.flat(dW0_out, w0_shared ? state : states, true);
    if (k.st != TTT_OK) return k.st;
    const size_t need = backward_ws_bytes(c.d, c.fp32);
    if (!ws || ws_bytes < need) return TTT_ERR_WORKSPACE;
    if (misaligned(ws, 256)) return TTT_ERR_ALIGNMENT;
    k.flat(ws, (long long)need, true);
    st = k.finish();
    if (st != TTT_OK) return st;
    c.W0 = W0;
    c.w0_bs = w0_shared ? 0 : state / 4;
    c.dW1 = dW1;
    c.dW0 = dW0_out;
    c.ws = static_cast<uint8_t*>(ws);
    c.wait_ns = wait_limit_ns();
    c.sms = sm_count();
    c.stream = static_cast<cudaStream_t>(stream);
    return launch_backward(c);
}

ttt_status ttt_step_gated_delta(const ttt_view* Q, const ttt_view* K, const ttt_view* V, const ttt_view* G, const ttt_view* Beta,
                                float* W, int n_slots, const int* slots, float scale, const ttt_view* Z, const ttt_delta_shape* s,
                                void* stream) {
    ttt_status st = check_delta_shape(s);
    if (st != TTT_OK) return st;
    if (!std::isfinite(scale) || n_slots < 1 || !W) return TTT_ERR_INVALID_ARG;
    if (!slots && n_slots < s->batch) return TTT_ERR_INVALID_ARG;
    if ((long long)s->batch * s->heads * (s->d_v / 16) > (1LL << 31) - 1) return TTT_ERR_UNSUPPORTED;
    gd::Call c{};
    c.d = dims_of(*s);
    c.fp32 = s->dtype == TTT_FP32;
    c.d.scale = scale;
    Arguments k{s};
    k.tokens(Q, s->qk_heads, s->d_k, &c.Q, false);
    k.tokens(K, s->qk_heads, s->d_k, &c.K, false);
    k.tokens(V, s->heads, s->d_v, &c.V, false);
    k.tokens(G, s->heads, 1, &c.G, false, true);
    k.tokens(Beta, s->heads, 1, &c.Beta, false, true);
    k.tokens(Z, s->heads, s->d_v, &c.Z, true);
    k.flat(slots, 4LL * s->batch, false, 4);
    k.flat(W, (long long)n_slots * s->heads * s->d_v * s->d_k * 4, true);
    st = k.finish();
    if (st != TTT_OK) return st;
    c.sms = sm_count();
    c.stream = static_cast<cudaStream_t>(stream);
    return launch_step(c, W, slots, n_slots);
}

size_t ttt_clip_workspace_bytes(int n) { return n < 1 ? 0 : clip_ws_bytes(n); }

ttt_status ttt_clip_gradients(const void* const* grads, void* const* out, const long long* counts, const int* dtypes, int n,
                              float max_norm, float* norm_out, void* ws, size_t ws_bytes, void* stream) {
    if (n < 1 || !grads || !out || !counts || !dtypes || !norm_out) return TTT_ERR_INVALID_ARG;
    if (!(max_norm >= 0.f)) return TTT_ERR_INVALID_ARG;
    if (!ws || ws_bytes < clip_ws_bytes(n)) return TTT_ERR_WORKSPACE;
    if (misaligned(ws, 256) || misaligned(norm_out, 4)) return TTT_ERR_ALIGNMENT;
    struct Span {
        const char *lo, *hi;
        int index;
        bool write;
    };
    Span* spans = new (std::nothrow) Span[2 * (size_t)n + 2];
    if (!spans) return TTT_ERR_INVALID_ARG;
    int m = 0;
    ttt_status st = TTT_OK;
    auto span = [&](const void* p, long long bytes, int index, bool write) {
        spans[m++] = Span{static_cast<const char*>(p), static_cast<const char*>(p) + bytes, index, write};
    };
    for (int i = 0; i < n && st == TTT_OK; ++i) {
        if (dtypes[i] != TTT_FP32 && dtypes[i] != TTT_BF16) st = TTT_ERR_INVALID_ARG;
        else if (counts[i] < 0 || counts[i] > (1LL << 40)) st = TTT_ERR_INVALID_ARG;
        else if (counts[i] > 0) {
            const int es = dtypes[i] == TTT_FP32 ? 4 : 2;
            if (!grads[i] || !out[i]) st = TTT_ERR_INVALID_ARG;
            else if (misaligned(grads[i], es) || misaligned(out[i], es)) st = TTT_ERR_ALIGNMENT;
            else {
                span(out[i], counts[i] * es, i, true);
                if (out[i] != grads[i]) span(grads[i], counts[i] * es, i, false);
            }
        }
    }
    if (st == TTT_OK) {
        span(ws, (long long)clip_ws_bytes(n), n, true);
        span(norm_out, 4, n + 1, true);
        std::sort(spans, spans + m, [](const Span& a, const Span& b) { return a.lo < b.lo; });
        const int dev = current_device();
        const char *end_any = nullptr, *end_write = nullptr;    // furthest end seen, of any span and of an output
        for (int i = 0; i < m && st == TTT_OK; ++i) {
            if (spans[i].lo < (spans[i].write ? end_any : end_write)) st = TTT_ERR_INVALID_ARG;
            end_any = std::max(end_any, spans[i].hi);
            if (spans[i].write) end_write = std::max(end_write, spans[i].hi);
        }
        for (int i = 0; i < m && st == TTT_OK; ++i)
            if (!device_ptr(spans[i].lo, dev)) st = TTT_ERR_INVALID_ARG;
    }
    delete[] spans;
    if (st == TTT_OK) st = ttt_last_error();
    if (st != TTT_OK) return st;
    return launch_clip(grads, out, counts, dtypes, n, max_norm, norm_out, ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
