// delta.cuh -- host-side description of a gated-delta call and the device helpers its kernels share:
// warp-level bf16 matrix products (mma.sync m16n8k16, fp32 accumulation), ldmatrix / stmatrix, 16-byte
// asynchronous copies, and the split of an fp32 value into bf16 parts.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sm100.cuh"
#include "ttt_internal.h"

namespace ttt {
namespace gd {

constexpr int CT = 32;                // tokens per chunk of the sequential kernels
constexpr int MP = CT + 8;            // row pitch (elements) of a 32 x 32 bf16 matrix image

// Strided [batch][heads][tokens][width] view, unit stride along the width.
struct View {
    char* p;
    long long bs, hs, ts;             // strides in elements
};
// A view whose values are sums of bf16 parts, `ps` elements apart (a bf16 tensor has one part).
struct Parts {
    const __nv_bfloat16* p;
    long long ps, bs, hs, ts;
};

struct Dims {
    int B, hk, h, r, N, dk, dv;       // r = h / hk value heads per key head
    int nc;                           // chunks of CT tokens per sequence
    int ng, gt;                       // groups of gt tokens per sequence (backward)
    const int* lengths;               // nullable [B]
    float scale;
};

// bf16 parts of an operand that no bf16 value holds: 24 bits, as many as fp32 has.
constexpr int P = 3;
// Per (image, value head, chunk) record in the workspace, written by the prep kernel and copied as it
// is into shared memory: gates (gamma, suffix, beta), then the part images of T', A and (backward) T_u.
constexpr int kGateBytes = 3 * CT * 4;
constexpr int kMat = P * CT * MP * 2;
__host__ __device__ constexpr int rec_bytes(bool backward) { return kGateBytes + (backward ? 3 : 2) * kMat; }

struct Call {
    Dims d;
    bool fp32;
    View Q, K, V, Z;                  // Z: forward output, or dZ in the backward pass
    View G, Beta;                     // fp32 [B][h][N] (hs, ts, bs used)
    const float* W0;                  // nullable
    long long w0_bs;                  // 0: shared by the batch
    float* W1_out;                    // nullable (forward)
    const float* dW1;                 // nullable (backward)
    View dQ, dK, dV, dG, dBeta;
    float* dW0;                       // nullable: dW0 of the layout of W0
    uint8_t* ws;                      // starts with a header whose first word is the error word
    cudaStream_t stream;
    unsigned long long wait_ns;       // bound of every device-side wait (ns)
    int sms;                          // SMs of the device
};

size_t forward_ws_bytes(const Dims& d, bool fp32);
size_t backward_ws_bytes(const Dims& d, bool fp32);
ttt_status launch_forward(const Call& c);
ttt_status launch_backward(const Call& c);
ttt_status launch_step(const Call& c, float* W, const int* slots, int n_slots);
// Group size (tokens) of the backward pass's parallel kernel.
inline int group_tokens(bool fp32) { return fp32 ? 32 : 64; }

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t s32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r0), "r"(r1), "r"(r2),
                 "r"(r3)
                 : "memory");
}
// How long a CTA that gives up waits for its own copies and products: 50 ms at least, however short the call's limit, since what
// lands after its end lands in another CTA's memory.
__device__ __forceinline__ unsigned long long drain_limit(const Abort& ab) { return max(ab.limit, 50000000ull); }

// D (16 x 8, fp32) += A (16 x 16, bf16) * B (16 x 8, bf16).
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// (x, y) as P packed bf16 pairs whose sum is (x, y) up to 2^-24 relative: part 0 is the nearest bf16,
// part p the nearest bf16 to what the earlier parts leave.  (An infinite value gives NaN parts: a state
// that overflowed ends in NaN.)
__device__ __forceinline__ void split2(float x, float y, uint32_t (&o)[P]) {
    o[0] = pack2(x, y);
#pragma unroll
    for (int p = 1; p < P; ++p) {
        x -= lo_f(o[p - 1]);
        y -= hi_f(o[p - 1]);
        o[p] = pack2(x, y);
    }
}

// Sequence length of image b, clamped to the padded length.
__device__ __forceinline__ int seq_len(const Dims& d, int b) {
    return d.lengths ? max(0, min(d.N, d.lengths[b])) : d.N;
}
#endif

}  // namespace gd
}  // namespace ttt
