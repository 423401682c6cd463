// clip.cu -- the global norm of many tensors and their scaling to a largest norm:
//   n = sqrt(sum over all tensors of x^2),   out = x min(1, max_norm / n).
//
// Two launches for up to kTable tensors (two more for each kTable beyond): the first reads every tensor once and
// leaves one partial sum per CTA, the second starts by adding those up (the same order in every CTA, so
// that all use the same factor) and scales.  The tensors' addresses travel as a kernel argument, so that
// nothing is copied to the device and a captured graph holds all it needs.
//
// Bound: HBM, one read for the norm, then one read and one write.  The second pass walks the tensors backwards:
// what the first read last is still in L2 (126 MB) and is read from there.  667 MB of bf16 and fp32 gradients in 60
// tensors: 338 to 350 us, 5.8 TB/s counting both reads.  60 tensors of 400,000 elements in all: 25 us, the host's (its checks of each
// tensor and two launches).  Sums: fp32 over the 4 or 8
// values of a 16-byte piece (fp64 where their squares leave fp32's range), then fp64; fixed order.
#include <algorithm>

#include "delta.cuh"

namespace ttt {
namespace clip {

constexpr int kTable = 256;               // tensors per launch (a small table for up to kSmall: less to pass)
constexpr int kSmall = 64;
constexpr int kThreads = 256;
constexpr int kLoads = 8;                 // 16-byte loads a thread has in flight
constexpr int kPiece = kThreads * 16 * kLoads;   // bytes of a tensor that a CTA takes at a time
// 32 for each of a B200's SMs, several waves: 377 us with as many as fit at a time, 341 us with these (667 MB of gradients).  Sizes the workspace.
constexpr int kMaxCtas = 148 * 32;

struct Item {
    const char* in;
    char* out;
    long long bytes;                      // of the tensor
    int first;                            // first piece (over the launch's tensors)
    int fp32;
};
template <int M>
struct Table {
    Item it[M];
    int n, pieces;
};

template <int M>
__device__ __forceinline__ int find_item(const Table<M>& t, int piece) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.it[mid].first <= piece) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A piece of a tensor: bytes [lo, hi) from its start; [vlo, vhi) the 16-byte aligned part of the input.
struct Range {
    long long lo, vlo, vhi, hi;
};
__device__ __forceinline__ Range range_of(const Item& it, int piece) {
    const long long head = min((long long)((16 - (reinterpret_cast<uintptr_t>(it.in) & 15)) & 15), it.bytes);
    const long long k = piece - it.first;
    Range r;
    r.vlo = min(head + k * kPiece, it.bytes);
    r.lo = k == 0 ? 0 : r.vlo;
    r.hi = min(head + (k + 1) * kPiece, it.bytes);
    r.vhi = r.vlo + (r.hi - r.vlo) / 16 * 16;
    return r;
}

// The sum of a 16-byte piece's squares.  Squares that overflow fp32, or that lose bits or vanish below its
// normal range, are taken again in fp64.
__device__ __forceinline__ double sq_piece(uint4 w, int fp32) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (fp32) s = fmaf(__uint_as_float(x[i]), __uint_as_float(x[i]), s);
        else s = fmaf(gd::lo_f(x[i]), gd::lo_f(x[i]), fmaf(gd::hi_f(x[i]), gd::hi_f(x[i]), s));
    }
    if (s > 1e-28f && s < 3e38f) return (double)s;
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double a = fp32 ? __uint_as_float(x[i]) : gd::lo_f(x[i]), b = fp32 ? 0.f : gd::hi_f(x[i]);
        z += a * a + b * b;
    }
    return z;
}
__device__ __forceinline__ float one_at(const char* p, int fp32) {
    return fp32 ? *reinterpret_cast<const float*>(p) : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}

__device__ __forceinline__ double block_sum(double x, double* sm) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(~0u, x, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) x += sm[w];
    __syncthreads();
    return x;
}

template <int M>
__global__ void __launch_bounds__(kThreads) clip_norm(const __grid_constant__ Table<M> t, double* partial) {
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ double sm[kThreads / 32];
    double acc = 0.0;
    for (int piece = blockIdx.x; piece < t.pieces; piece += gridDim.x) {
        const Item& it = t.it[find_item(t, piece)];
        const Range r = range_of(it, piece);
        uint4 w[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const long long o = r.vlo + ((long long)i * kThreads + threadIdx.x) * 16;
            w[i] = o < r.vhi ? *reinterpret_cast<const uint4*>(it.in + o) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (w[i].x | w[i].y | w[i].z | w[i].w) acc += sq_piece(w[i], it.fp32);
        const int es = it.fp32 ? 4 : 2, heads = (int)(r.vlo - r.lo) / es, tails = (int)(r.hi - r.vhi) / es;
        if ((int)threadIdx.x < heads + tails) {        // fewer than 16 elements that no vector covers
            const int x = threadIdx.x;
            const float v = one_at(it.in + (x < heads ? r.lo + (long long)x * es : r.vhi + (long long)(x - heads) * es), it.fp32);
            acc += (double)v * v;
        }
    }
    acc = block_sum(acc, sm);
    if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

template <int M>
__global__ void __launch_bounds__(kThreads)
clip_scale(const __grid_constant__ Table<M> t, const double* partial, int n_partial, float max_norm, float* norm_out) {
    __shared__ double sm[kThreads / 32];
    pdl_wait_primary();
    double acc = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += kThreads) acc += partial[i];
    const double norm = sqrt(block_sum(acc, sm));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    // a NaN norm makes the factor NaN; an infinite one makes it zero
    const float f = norm <= (double)max_norm ? 1.f : (float)((double)max_norm / norm);
    for (int piece = t.pieces - 1 - blockIdx.x; piece >= 0; piece -= gridDim.x) {
        const Item& it = t.it[find_item(t, piece)];
        if (f == 1.f && it.in == it.out) continue;
        const Range r = range_of(it, piece);
        const int es = it.fp32 ? 4 : 2;
        const bool vec = ((reinterpret_cast<uintptr_t>(it.in) ^ reinterpret_cast<uintptr_t>(it.out)) & 15) == 0;
        uint4 w[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const long long o = r.vlo + ((long long)i * kThreads + threadIdx.x) * 16;
            if (o < r.vhi) w[i] = __ldcs(reinterpret_cast<const uint4*>(it.in + o));
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const long long o = r.vlo + ((long long)i * kThreads + threadIdx.x) * 16;
            if (o >= r.vhi) continue;
            uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            if (it.fp32) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = gd::pack2(gd::lo_f(x[j]) * f, gd::hi_f(x[j]) * f);
            }
            char* out = it.out + o;
            if (vec) {
                __stcs(reinterpret_cast<uint4*>(out), make_uint4(x[0], x[1], x[2], x[3]));
            } else if (it.fp32) {
#pragma unroll
                for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(out)[j] = x[j];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    reinterpret_cast<uint16_t*>(out)[2 * j] = (uint16_t)x[j];
                    reinterpret_cast<uint16_t*>(out)[2 * j + 1] = (uint16_t)(x[j] >> 16);
                }
            }
        }
        const int heads = (int)(r.vlo - r.lo) / es, tails = (int)(r.hi - r.vhi) / es;
        if ((int)threadIdx.x < heads + tails) {
            const int x = threadIdx.x;
            const long long o = x < heads ? r.lo + (long long)x * es : r.vhi + (long long)(x - heads) * es;
            const float v = one_at(it.in + o, it.fp32) * f;
            if (it.fp32) *reinterpret_cast<float*>(it.out + o) = v;
            else *reinterpret_cast<__nv_bfloat16*>(it.out + o) = __float2bfloat16_rn(v);
        }
    }
}

static int pieces_of(const void* in, long long bytes) {
    const long long head = std::min<long long>((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15, bytes);
    return (int)std::max<long long>(bytes > 0 ? 1 : 0, (bytes - head + kPiece - 1) / kPiece);
}

}  // namespace clip

size_t clip_ws_bytes(int n) {
    return (size_t)((n + clip::kTable - 1) / clip::kTable) * clip::kMaxCtas * sizeof(double);
}

template <int M>
static ttt_status launch_clip_t(const void* const* in, void* const* out, const long long* counts, const int* dtypes, int n, float max_norm,
                                float* norm_out, double* partial, cudaStream_t st) {
    using namespace clip;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;      // each kernel waits for the one before it
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int used = 0;
    for (int pass = 0; pass < 2; ++pass)
        for (int t0 = 0, seg = 0; t0 < n; t0 += M, ++seg) {
            Table<M> t;
            t.n = 0;
            t.pieces = 0;
            for (int i = t0; i < std::min(n, t0 + M); ++i) {
                const int es = dtypes[i] == TTT_FP32 ? 4 : 2;
                const long long bytes = counts[i] * es;
                if (bytes == 0) continue;
                t.it[t.n++] = Item{static_cast<const char*>(in[i]), static_cast<char*>(out[i]), bytes, t.pieces, dtypes[i] == TTT_FP32};
                t.pieces += pieces_of(in[i], bytes);
            }
            const int grid = std::max(1, std::min(t.pieces, kMaxCtas));
            cfg.gridDim = dim3(grid);
            cudaError_t e;
            if (pass == 0) {
                e = cudaLaunchKernelEx(&cfg, clip_norm<M>, t, partial + used);
                used += grid;
            } else {
                e = cudaLaunchKernelEx(&cfg, clip_scale<M>, t, (const double*)partial, used, max_norm, seg == 0 ? norm_out : (float*)nullptr);
            }
            const ttt_status s = check_launch(e);
            if (s != TTT_OK) return s;
        }
    return TTT_OK;
}

ttt_status launch_clip(const void* const* in, void* const* out, const long long* counts, const int* dtypes, int n, float max_norm,
                       float* norm_out, void* ws, cudaStream_t st) {
    double* partial = static_cast<double*>(ws);
    return n <= clip::kSmall ? launch_clip_t<clip::kSmall>(in, out, counts, dtypes, n, max_norm, norm_out, partial, st)
                             : launch_clip_t<clip::kTable>(in, out, counts, dtypes, n, max_norm, norm_out, partial, st);
}

}  // namespace ttt
