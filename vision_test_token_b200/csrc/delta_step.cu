// delta_step.cu -- the gated delta rule's recurrent form: a few tokens (one, or a few drafted ones) of
// each sequence of a batch, on a cache of fp32 states that is updated in place.
//
// With the old state W of a row of the state matrix, a = W.k, c = W.q and the gate f = e^g:
//   u = beta (v - f a),   z = scale (f c + u (k.q)),   W <- f W + u k,
// so that both dot products use the state as it was read and one pass over it is enough.
//
// Bound: HBM.  A state is read once and written once (2 x 4 dk dv bytes per sequence and head, about
// 130 times a token's own rows).  Eight lanes share a row (128 contiguous bytes per load), so a dot product
// takes three shuffles; a thread holds the pieces of 1 or 4 rows (RPT), all loads in flight before the first use.
// 247 sequences with 32 heads of 128 x 128: 162 us, 6.4 TB/s.
#include "delta.cuh"

namespace ttt {
namespace gd {

struct StepArgs {
    Dims d;
    View Q, K, V, G, Beta, Z;
    float* W;                     // [n_slots][h][dv][dk]
    const int* slots;             // nullable [B]
    int n_slots;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(lo_f(w.x), hi_f(w.x), lo_f(w.y), hi_f(w.y));
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(~0u, x, 4);
    x += __shfl_xor_sync(~0u, x, 2);
    return x + __shfl_xor_sync(~0u, x, 1);
}

template <typename E, int DK, int RPT>
__global__ void __launch_bounds__(128) delta_step(StepArgs s) {
    constexpr int NV = DK / 32;                       // float4 pieces of a row per lane
    constexpr int ROWS = 16 * RPT;
    const Dims& d = s.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 3, p = lane & 7;
    const int slices = d.dv / ROWS;
    const int slice = blockIdx.x % slices;
    const int h = blockIdx.x / slices % d.h;
    int b = blockIdx.x / slices / d.h;
    const int slot = s.slots ? s.slots[b] : b;
    if (slot < 0 || slot >= s.n_slots) return;        // an unused row of the batch
    const int row0 = slice * ROWS + warp * 4 * RPT + r;
    float* W = s.W + ((long long)slot * d.h + h) * d.dv * DK + (long long)row0 * DK + p * 4;
    float4 w[RPT][NV];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
#pragma unroll
        for (int i = 0; i < NV; ++i) w[m][i] = load4(W + m * 4 * DK + i * 32);

    // Rows of the batch that name the same state take their steps in batch order, on this CTA: the first
    // of them owns the state.
    __shared__ int next_of[4];
    auto later = [&](int from, bool* owned) {         // first row after `from` with this slot, B if none
        int first = d.B;
        bool earlier = false;
        for (int x = tid; x < d.B; x += 128) {
            if (x == from || s.slots[x] != slot) continue;
            if (x < from) earlier = true;
            else first = min(first, x);
        }
        first = __reduce_min_sync(~0u, first);
        if (lane == 0) next_of[warp] = first;
        const bool any = __syncthreads_or(earlier);
        if (owned) *owned = any;
        first = min(min(next_of[0], next_of[1]), min(next_of[2], next_of[3]));
        __syncthreads();
        return first;
    };
    int next = d.B;
    if (s.slots) {
        bool owned;
        next = later(b, &owned);
        if (owned) return;
    }

    for (;;) {
        const int hk = h / d.r;
        for (int t = 0; t < d.N; ++t) {
            const E* kp = reinterpret_cast<const E*>(s.K.p) + b * s.K.bs + hk * s.K.hs + t * s.K.ts + p * 4;
            const E* qp = reinterpret_cast<const E*>(s.Q.p) + b * s.Q.bs + hk * s.Q.hs + t * s.Q.ts + p * 4;
            const E* vp = reinterpret_cast<const E*>(s.V.p) + b * s.V.bs + h * s.V.hs + t * s.V.ts + row0;
            float4 k[NV], q[NV];
            float v[RPT];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                k[i] = load4(kp + i * 32);
                q[i] = load4(qp + i * 32);
            }
#pragma unroll
            for (int m = 0; m < RPT; ++m) v[m] = load1(vp + m * 4);
            const float f = expf(reinterpret_cast<const float*>(s.G.p)[b * s.G.bs + h * s.G.hs + t * s.G.ts]);
            const float beta = reinterpret_cast<const float*>(s.Beta.p)[b * s.Beta.bs + h * s.Beta.hs + t * s.Beta.ts];
            float kq = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) kq = dot4(k[i], q[i], kq);
            kq = sum8(kq);
            E* zp = reinterpret_cast<E*>(s.Z.p) + b * s.Z.bs + h * s.Z.hs + t * s.Z.ts + row0;
#pragma unroll
            for (int m = 0; m < RPT; ++m) {
                float a = 0.f, c = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    a = dot4(w[m][i], k[i], a);
                    c = dot4(w[m][i], q[i], c);
                }
                a = sum8(a);
                c = sum8(c);
                const float u = beta * fmaf(-f, a, v[m]);
                if (p == 0) store1(zp + m * 4, d.scale * fmaf(f, c, u * kq));
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    w[m][i].x = fmaf(u, k[i].x, f * w[m][i].x);
                    w[m][i].y = fmaf(u, k[i].y, f * w[m][i].y);
                    w[m][i].z = fmaf(u, k[i].z, f * w[m][i].z);
                    w[m][i].w = fmaf(u, k[i].w, f * w[m][i].w);
                }
            }
        }
        if (next >= d.B) break;
        b = next;
        next = later(b, nullptr);
    }
#pragma unroll
    for (int m = 0; m < RPT; ++m)
#pragma unroll
        for (int i = 0; i < NV; ++i) *reinterpret_cast<float4*>(W + m * 4 * DK + i * 32) = w[m][i];
}

template <typename E, int DK>
static ttt_status step_t(const StepArgs& s, int sms, cudaStream_t st) {
    const long long rows = (long long)s.d.B * s.d.h * s.d.dv;
    // One row per thread spreads a small batch over more SMs, four have more loads in flight.  Heads of 128 x 128, one
    // row against four: 32 heads 2.5 / 2.7 us, 512 heads 13.3 / 13.4, 1024 heads 24.6 / 23.8, 8192 heads 225 / 161.
    if (rows >= 512LL * sms)
        delta_step<E, DK, 4><<<(unsigned)(rows / 64), 128, 0, st>>>(s);
    else
        delta_step<E, DK, 1><<<(unsigned)(rows / 16), 128, 0, st>>>(s);
    return check_launch(cudaGetLastError());
}

ttt_status launch_step(const Call& c, float* W, const int* slots, int n_slots) {
    const StepArgs s{c.d, c.Q, c.K, c.V, c.G, c.Beta, c.Z, W, slots, n_slots};
    if (c.fp32) return c.d.dk == 64 ? step_t<float, 64>(s, c.sms, c.stream) : step_t<float, 128>(s, c.sms, c.stream);
    return c.d.dk == 64 ? step_t<__nv_bfloat16, 64>(s, c.sms, c.stream) : step_t<__nv_bfloat16, 128>(s, c.sms, c.stream);
}

}  // namespace gd
}  // namespace ttt
