// delta.cu -- the gated delta rule over whole sequences: forward pass and the states it passes through.
//
//   W_t = e^{g_t} W_{t-1} + beta_t (v_t - e^{g_t} W_{t-1} k_t) k_t^T,   z_t = scale W_t q_t
//
// Chunks of C = 32 tokens.  With gamma_i = exp(g_1 + .. + g_i) inside a chunk, Gamma_ij = exp(g_{j+1} + .. +
// g_i) for j <= i and G_ij = Gamma_ij k_i.k_j for j < i, the residuals e_i = v_i - e^{g_i} W_{i-1} k_i of a
// chunk that starts from W solve (I + G diag(beta)) E = V - diag(gamma) K W^T.  So
//   prep   (one warp per image, value head and chunk, all at once):
//          T' = (I + G diag(beta))^{-1} by forward substitution, A = scale Gamma .* (Q K^T) for j <= i;
//   chain  (one warp per 16 rows of W, sequential over the chunks):
//          R = V - diag(gamma) K W^T,  E = T' R,  U = diag(beta) E,
//          Z = scale diag(gamma) Q W^T + A U,   W <- gamma_C W + U^T diag(Gamma_C.) K.
// Every sum of log gates starts at zero (no difference of two long prefix sums), so a gate of -inf
// (a state that is dropped) and strong gates keep their accuracy.
//
// The chain's rows are independent, so that a warp that owns 16 rows of W keeps them in registers as
// the accumulators of U^T K, and each product's accumulators are the next one's left operand (the
// m16n8k16 accumulator and A-operand layouts agree after a pack to bf16): W -> K W^T -> E -> W never
// touches shared memory and no warp waits on another within a chunk.
//
// Precision: W is fp32.  As an operand it is split into P bf16 parts (2 for bf16 tokens: about 16
// significant bits; 3 for fp32 tokens: about 24), as are R, E, U, T' and A; bf16 tokens are exact
// operands, fp32 tokens are split into 3 parts by a pass of their own.  Products of parts below the last
// kept part are dropped.
//
// Bound: the chain of chunks (per chunk and warp about 300 matrix instructions at d = 128, issued one per
// 8 cycles per SM quarter: the instruction's rate here was measured at 1,009 multiply-adds per cycle and SM).
#include <algorithm>

#include "delta.cuh"

namespace ttt {
namespace gd {

// --------------------------------------------------------------------------------------------------
// fp32 tokens -> bf16 parts, contiguous [part][B][heads][N][width]
// --------------------------------------------------------------------------------------------------
template <int P>
__global__ void split_tokens(View x, __nv_bfloat16* out, long long ps, int heads, int N, int width, long long total4) {
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total4; i += (long long)gridDim.x * blockDim.x) {
        const int w4 = width / 4;
        const int c = (int)(i % w4) * 4;
        const long long row = i / w4;
        const int t = (int)(row % N);
        const long long bh = row / N;
        const int h = (int)(bh % heads), b = (int)(bh / heads);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x.p) + b * x.bs + h * x.hs + t * x.ts + c);
        uint32_t lo[P], hi[P];
        split2<P>(v.x, v.y, lo);
        split2<P>(v.z, v.w, hi);
#pragma unroll
        for (int p = 0; p < P; ++p) *reinterpret_cast<uint2*>(out + p * ps + row * width + c) = make_uint2(lo[p], hi[p]);
    }
}

// --------------------------------------------------------------------------------------------------
// Prep
// --------------------------------------------------------------------------------------------------
constexpr int GP = CT + 4;            // row pitch (floats) of the 32 x 32 fp32 matrices of a warp

// Warps (chunks) per CTA: as many as leave room for a second CTA on the SM (bf16), or fit (fp32 parts).
template <int DK, int PK>
__host__ __device__ constexpr int prep_warps() { return PK == 1 ? 4 : 2; }

template <int DK, int PK>
__host__ __device__ constexpr int prep_tile_bytes() { return PK * CT * (DK + 8) * 2; }
template <int DK, int PK>
__host__ __device__ constexpr int prep_warp_bytes() { return 2 * prep_tile_bytes<DK, PK>() + 2 * CT * GP * 4; }

// 32 tokens x 32 tokens of X Y^T over DK features; X, Y [part][32][DK + 8].  Two 16-row tiles.
template <int DK, int PK>
__device__ __forceinline__ void gram32(float (&c)[2][4][4], uint32_t x, uint32_t y, int lane) {
    constexpr int KP = DK + 8, PB = CT * KP * 2;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) c[m][n][q] = 0.f;
    const int mi = lane >> 3, lr = lane & 7;
    const uint32_t aoff = (((mi & 1) * 8 + lr) * KP + (mi >> 1) * 8) * 2;
    const uint32_t boff = (((mi >> 1) * 8 + lr) * KP + (mi & 1) * 8) * 2;
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) {
        uint32_t b[PK][2][4];
#pragma unroll
        for (int p = 0; p < PK; ++p)
#pragma unroll
            for (int n2 = 0; n2 < 2; ++n2) ldsm4(b[p][n2], y + p * PB + boff + (n2 * 16 * KP + kk * 16) * 2);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int pa = 0; pa < PK; ++pa) {
                uint32_t a[4];
                ldsm4(a, x + pa * PB + aoff + (m * 16 * KP + kk * 16) * 2);
#pragma unroll
                for (int pb = 0; pa + pb < PK; ++pb)
#pragma unroll
                    for (int n2 = 0; n2 <= m; ++n2) {        // the upper triangle is not used
                        mma16816(c[m][2 * n2], a, b[pb][n2][0], b[pb][n2][1]);
                        mma16816(c[m][2 * n2 + 1], a, b[pb][n2][2], b[pb][n2][3]);
                    }
            }
        }
    }
}

__device__ __forceinline__ void put32(float* dst, const float (&c)[2][4][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            *reinterpret_cast<float2*>(dst + (m * 16 + g) * GP + n * 8 + 2 * t) = make_float2(c[m][n][0], c[m][n][1]);
            *reinterpret_cast<float2*>(dst + (m * 16 + g + 8) * GP + n * 8 + 2 * t) = make_float2(c[m][n][2], c[m][n][3]);
        }
}

// Row i, column `lane` of a bf16 part image.
template <int P>
__device__ __forceinline__ void put_part(uint8_t* mat, int i, int lane, float x) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const __nv_bfloat16 v = __float2bfloat16_rn(x);
        reinterpret_cast<__nv_bfloat16*>(mat)[(p * CT + i) * MP + lane] = v;
        x -= __bfloat162float(v);
    }
}

template <int DK, int P, int PK, bool BACKWARD>
__global__ void __launch_bounds__(prep_warps<DK, PK>() * 32)
delta_prep(Dims d, Parts Q, Parts K, View G, View Beta, uint8_t* rec, long long total) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int KP = DK + 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long item = (long long)blockIdx.x * prep_warps<DK, PK>() + warp;
    if (item >= total) return;
    const int c = (int)(item % d.nc);
    const long long bh = item / d.nc;
    const int h = (int)(bh % d.h), b = (int)(bh / d.h);
    const int left = seq_len(d, b) - c * CT;
    if (left <= 0) return;
    uint8_t* my = smem + warp * prep_warp_bytes<DK, PK>();
    const uint32_t kt = s32(my), qt = kt + prep_tile_bytes<DK, PK>();
    float* kkm = reinterpret_cast<float*>(my + 2 * prep_tile_bytes<DK, PK>());
    float* qkm = kkm + CT * GP;
    {
        const long long ko = b * K.bs + (h / d.r) * K.hs + (long long)c * CT * K.ts;
        const long long qo = b * Q.bs + (h / d.r) * Q.hs + (long long)c * CT * Q.ts;
        constexpr int CPR = DK / 8;
#pragma unroll
        for (int p = 0; p < PK; ++p)
#pragma unroll 4
            for (int x = lane; x < CT * CPR; x += 32) {
                const int row = x / CPR, col = x % CPR;
                const bool live = row < left;
                const long long rk = live ? row : 0;
                cp16(kt + (p * CT * KP + row * KP + col * 8) * 2, K.p + p * K.ps + ko + rk * K.ts + col * 8, live);
                cp16(qt + (p * CT * KP + row * KP + col * 8) * 2, Q.p + p * Q.ps + qo + rk * Q.ts + col * 8, live);
            }
        cp_commit();
    }
    // gates of token `lane`; tokens past the end of the sequence neither fade nor write
    const long long t = (long long)c * CT + lane;
    const bool live = lane < left;
    const float g = live ? reinterpret_cast<const float*>(G.p)[b * G.bs + h * G.hs + t * G.ts] : 0.f;
    const float beta = live ? reinterpret_cast<const float*>(Beta.p)[b * Beta.bs + h * Beta.hs + t * Beta.ts] : 0.f;
    float pre = g, suf = __shfl_down_sync(~0u, g, 1);
    if (lane == 31) suf = 0.f;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const float a = __shfl_up_sync(~0u, pre, o), z = __shfl_down_sync(~0u, suf, o);
        if (lane >= o) pre += a;
        if (lane + o < 32) suf += z;
    }
    uint8_t* out = rec + item * rec_bytes(P, BACKWARD);
    float* gates = reinterpret_cast<float*>(out);
    gates[lane] = expf(pre);
    gates[CT + lane] = expf(suf);
    gates[2 * CT + lane] = beta;

    cp_wait<0>();
    __syncwarp();
    {
        float m[2][4][4];
        gram32<DK, PK>(m, kt, kt, lane);
        put32(kkm, m, lane);
        gram32<DK, PK>(m, qt, kt, lane);
        put32(qkm, m, lane);
    }
    __syncwarp();
    // column `lane` (= j): Gamma_ij with its log summed from zero at i = j
    uint8_t* Tm = out + kGateBytes;
    uint8_t* Am = Tm + mat_bytes(P);
    uint8_t* Um = Am + mat_bytes(P);
    float s = 0.f;
#pragma unroll 4
    for (int i = 0; i < CT; ++i) {
        const float gi = __shfl_sync(~0u, g, i);
        s = i > lane ? s + gi : 0.f;
        const float dec = i >= lane ? expf(s) : 0.f;
        const float a = i >= lane ? d.scale * dec * qkm[i * GP + lane] : 0.f;
        put_part<P>(Am, i, lane, a);
        kkm[i * GP + lane] = i > lane ? dec * kkm[i * GP + lane] : 0.f;
    }
    __syncwarp();
    float y[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        float x = i == lane ? 1.f : 0.f;
#pragma unroll
        for (int l = 0; l < i; ++l) x = fmaf(-kkm[i * GP + l], y[l], x);
        put_part<P>(Tm, i, lane, x);
        y[i] = x * __shfl_sync(~0u, beta, i);
    }
    if constexpr (BACKWARD) {
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            float a = 0.f;
#pragma unroll
            for (int l = 0; l < i; ++l) a = fmaf(kkm[i * GP + l], y[l], a);
            const float x = (i == lane ? 1.f : 0.f) - __shfl_sync(~0u, beta, i) * a;
            put_part<P>(Um, i, lane, x);
            y[i] = x;
        }
    }
}

// --------------------------------------------------------------------------------------------------
// Chain
// --------------------------------------------------------------------------------------------------
struct ChainOut {
    View Z;                       // forward: the readout
    float* W1;                    // nullable [B][h][dv][dk]
    __nv_bfloat16* E;             // backward: residual parts [P][B][h][N][dv]
    long long e_ps;
    __nv_bfloat16* S;             // backward: states at the groups' starts [B][h][ng][P][dv][dk]
};

template <int DK, int P, int PK, int NW, bool SAVE>
struct ChainLayout {
    static constexpr int KP = DK + 8;
    static constexpr int VW = NW * 16;
    static constexpr int VE = PK == 1 ? 2 : 4;                 // bytes of a value element
    static constexpr int VP = PK == 1 ? VW + 8 : VW + 4;
    static constexpr int kK = PK * CT * KP * 2;
    static constexpr int kQ = SAVE ? 0 : kK;
    static constexpr int kV = CT * VP * VE;
    static constexpr int kR = kGateBytes + (SAVE ? 1 : 2) * mat_bytes(P);
    static constexpr int stage = kK + kQ + kV + kR;
    static constexpr int kStages = 3 * stage <= 110 * 1024 ? 3 : 2;
    static constexpr int warp_out = CT * 24 * 2;               // 32 tokens x 16 values, pitch 24
    static constexpr int smem = kStages * stage + NW * warp_out;
};

// One product step of the chain: acc[nb] += (parts a of 16 rows x 16 k) * B, nb = 0..3 (32 columns), B a
// matrix image [32][MP] with rows = columns of the product (n) and k contiguous; k block kk.
template <int P>
__device__ __forceinline__ void mat_nt(float (&acc)[4][4], const uint32_t (&a)[P][4], uint32_t mat, int kk, int lane) {
    const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
    for (int n2 = kk; n2 < 2; ++n2)                            // lower triangular: columns n >= k
#pragma unroll
        for (int pb = 0; pb < P; ++pb) {
            uint32_t b[4];
            ldsm4(b, mat + ((pb * CT + n2 * 16 + (mi >> 1) * 8 + lr) * MP + kk * 16 + (mi & 1) * 8) * 2);
#pragma unroll
            for (int pa = 0; pa + pb < P; ++pa) {
                mma16816(acc[2 * n2], a[pa], b[0], b[1]);
                mma16816(acc[2 * n2 + 1], a[pa], b[2], b[3]);
            }
        }
}

// The parts of accumulator blocks (2 kk, 2 kk + 1) as a left operand for k block kk.
template <int P>
__device__ __forceinline__ void as_operand(uint32_t (&a)[P][4], const float (&x)[4], const float (&y)[4]) {
    uint32_t o[P];
    split2<P>(x[0], x[1], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][0] = o[p];
    split2<P>(x[2], x[3], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][1] = o[p];
    split2<P>(y[0], y[1], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][2] = o[p];
    split2<P>(y[2], y[3], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][3] = o[p];
}

// s (16 x DK) += (parts a: 16 x 16 tokens of block kk) * X, X [part][32 tokens][DK + 8].
template <int DK, int P, int PK>
__device__ __forceinline__ void add_outer(float (&s)[DK / 8][4], const uint32_t (&a)[P][4], uint32_t x, int kk, int lane) {
    constexpr int KP = DK + 8;
    const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
    for (int n2 = 0; n2 < DK / 16; ++n2)
#pragma unroll
        for (int pb = 0; pb < PK; ++pb) {
            uint32_t b[4];
            ldsm4t(b, x + ((pb * CT + kk * 16 + (mi & 1) * 8 + lr) * KP + n2 * 16 + (mi >> 1) * 8) * 2);
#pragma unroll
            for (int pa = 0; pa + pb < P; ++pa) {
                mma16816(s[2 * n2], a[pa], b[0], b[1]);
                mma16816(s[2 * n2 + 1], a[pa], b[2], b[3]);
            }
        }
}

// acc (16 x 32 tokens) += (parts a: 16 x 16 features of block kk) * X^T, X [part][32 tokens][DK + 8].
template <int DK, int P, int PK>
__device__ __forceinline__ void dot_tokens(float (&acc)[4][4], const uint32_t (&a)[P][4], uint32_t x, int kk, int lane) {
    constexpr int KP = DK + 8;
    const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
    for (int n2 = 0; n2 < 2; ++n2)
#pragma unroll
        for (int pb = 0; pb < PK; ++pb) {
            uint32_t b[4];
            ldsm4(b, x + ((pb * CT + n2 * 16 + (mi >> 1) * 8 + lr) * KP + kk * 16 + (mi & 1) * 8) * 2);
#pragma unroll
            for (int pa = 0; pa + pb < P; ++pa) {
                mma16816(acc[2 * n2], a[pa], b[0], b[1]);
                mma16816(acc[2 * n2 + 1], a[pa], b[2], b[3]);
            }
        }
}

// 16 rows x 32 tokens held as accumulators -> bf16 rows [token][16] in `stage` (pitch 24) -> global rows.
__device__ __forceinline__ void put_rows(uint32_t stage, const uint32_t (&w)[8], __nv_bfloat16* dst, long long ts, int left,
                                         int lane) {
    const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
    for (int n2 = 0; n2 < 2; ++n2)
        stsm4t(stage + ((n2 * 16 + (mi >> 1) * 8 + lr) * 24 + (mi & 1) * 8) * 2, w[4 * n2], w[4 * n2 + 1], w[4 * n2 + 2],
               w[4 * n2 + 3]);
    __syncwarp();
    uint4 lo, hi;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w) : "r"(stage + lane * 48) : "memory");
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w) : "r"(stage + lane * 48 + 16) : "memory");
    if (lane < left) {
        uint4* o = reinterpret_cast<uint4*>(dst + lane * ts);
        o[0] = lo;
        o[1] = hi;
    }
    __syncwarp();
}

template <int P>
__device__ __forceinline__ void put_rows_parts(uint32_t stage, const float (&e)[4][4], __nv_bfloat16* dst, long long ps,
                                               long long ts, int left, int lane) {
    uint32_t w[P][8];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
        uint32_t o[P];
        split2<P>(e[nb][0], e[nb][1], o);
#pragma unroll
        for (int p = 0; p < P; ++p) w[p][2 * nb] = o[p];
        split2<P>(e[nb][2], e[nb][3], o);
#pragma unroll
        for (int p = 0; p < P; ++p) w[p][2 * nb + 1] = o[p];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) put_rows(stage, w[p], dst + p * ps, ts, left, lane);
}

// 16 rows x 32 tokens of accumulators -> the rows of a token tensor (bf16, or fp32 written directly:
// eight lanes hold eight consecutive features, a 32-byte sector).
template <int PK>
__device__ __forceinline__ void put_tokens(uint32_t stage, const float (&z)[4][4], char* base, long long off, long long ts, int left,
                                           int lane) {
    if constexpr (PK == 1) {
        uint32_t w[8];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            w[2 * nb] = pack2(z[nb][0], z[nb][1]);
            w[2 * nb + 1] = pack2(z[nb][2], z[nb][3]);
        }
        put_rows(stage, w, reinterpret_cast<__nv_bfloat16*>(base) + off, ts, left, lane);
    } else {
        const int g = lane >> 2, t = lane & 3;
        float* o = reinterpret_cast<float*>(base) + off;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int tok = nb * 8 + 2 * t + (q & 1);
                if (tok < left) o[tok * ts + g + (q >> 1) * 8] = z[nb][q];
            }
    }
}

// Rows [row0, row0 + 16) of the state [dv][dk] in global memory, as bf16 parts [P][dv][dk].
template <int DK, int P>
__device__ __forceinline__ void put_state_parts(const float (&s)[DK / 8][4], __nv_bfloat16* dst, int dv, int row0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const long long ps = (long long)dv * DK;
#pragma unroll
    for (int nb = 0; nb < DK / 8; ++nb)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t o[P];
            split2<P>(s[nb][2 * half], s[nb][2 * half + 1], o);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<uint32_t*>(dst + p * ps + (long long)(row0 + g + 8 * half) * DK + nb * 8 + 2 * t) = o[p];
        }
}
template <int DK>
__device__ __forceinline__ void put_state(const float (&s)[DK / 8][4], float* dst, int row0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nb = 0; nb < DK / 8; ++nb) {
        *reinterpret_cast<float2*>(dst + (long long)(row0 + g) * DK + nb * 8 + 2 * t) = make_float2(s[nb][0], s[nb][1]);
        *reinterpret_cast<float2*>(dst + (long long)(row0 + g + 8) * DK + nb * 8 + 2 * t) = make_float2(s[nb][2], s[nb][3]);
    }
}
template <int DK>
__device__ __forceinline__ void get_state(float (&s)[DK / 8][4], const float* src, int row0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nb = 0; nb < DK / 8; ++nb) {
        float2 a = make_float2(0.f, 0.f), b = a;
        if (src) {
            a = *reinterpret_cast<const float2*>(src + (long long)(row0 + g) * DK + nb * 8 + 2 * t);
            b = *reinterpret_cast<const float2*>(src + (long long)(row0 + g + 8) * DK + nb * 8 + 2 * t);
        }
        s[nb][0] = a.x; s[nb][1] = a.y; s[nb][2] = b.x; s[nb][3] = b.y;
    }
}

// 32 rows x W elements of E bytes into shared memory (row pitch in bytes), rows past `left` zero.
template <int W, int E, int NT>
__device__ __forceinline__ void load_rows(uint32_t dst, int pitch, const char* src, long long ts_bytes, int left, int tid) {
    constexpr int CPR = W * E / 16;
#pragma unroll
    for (int x0 = 0; x0 < CT * CPR; x0 += NT) {
        const int x = x0 + tid;
        if (CT * CPR % NT == 0 || x < CT * CPR) {
            const int row = x / CPR, col = x % CPR;
            const bool live = row < left;
            cp16(dst + row * pitch + col * 16, src + (live ? row : 0) * ts_bytes + col * 16, live);
        }
    }
}
template <int BYTES, int NT>
__device__ __forceinline__ void load_flat(uint32_t dst, const uint8_t* src, int tid) {
#pragma unroll
    for (int x0 = 0; x0 < BYTES / 16; x0 += NT) {
        const int x = x0 + tid;
        if (BYTES / 16 % NT == 0 || x < BYTES / 16) cp16(dst + x * 16, src + x * 16, true);
    }
}

__device__ __forceinline__ float2 lds2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds1(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <int DK, int P, int PK, int NW, bool SAVE>
__global__ void __launch_bounds__(NW * 32)
delta_chain(Dims d, Parts Q, Parts K, View V, const uint8_t* rec, const float* W0, long long w0_bs, ChainOut out) {
    using L = ChainLayout<DK, P, PK, NW, SAVE>;
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int NT = NW * 32, KP = L::KP;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int slices = d.dv / L::VW;
    const int slice = blockIdx.x % slices;
    const int bh = blockIdx.x / slices, b = bh / d.h, h = bh % d.h;
    const int len = seq_len(d, b), nch = (len + CT - 1) / CT;
    const int v0 = slice * L::VW, row0 = v0 + warp * 16;
    const uint32_t sb = s32(smem), wout = sb + L::kStages * L::stage + warp * L::warp_out;
    const int recb = rec_bytes(P, SAVE);

    auto issue = [&](int c) {
        if (c < nch) {
            const uint32_t st = sb + (c % L::kStages) * L::stage;
            const int left = len - c * CT;
            const long long tok = (long long)c * CT;
#pragma unroll
            for (int p = 0; p < PK; ++p) {
                load_rows<DK, 2, NT>(st + p * CT * KP * 2, KP * 2,
                                     reinterpret_cast<const char*>(K.p + p * K.ps + b * K.bs + (h / d.r) * K.hs + tok * K.ts),
                                     K.ts * 2, left, tid);
                if (!SAVE)
                    load_rows<DK, 2, NT>(st + L::kK + p * CT * KP * 2, KP * 2,
                                         reinterpret_cast<const char*>(Q.p + p * Q.ps + b * Q.bs + (h / d.r) * Q.hs + tok * Q.ts),
                                         Q.ts * 2, left, tid);
            }
            load_rows<L::VW, L::VE, NT>(st + L::kK + L::kQ, L::VP * L::VE,
                                        V.p + (b * V.bs + h * V.hs + tok * V.ts + v0) * L::VE, V.ts * L::VE, left, tid);
            load_flat<L::kR, NT>(st + L::kK + L::kQ + L::kV, rec + ((long long)bh * d.nc + c) * recb, tid);
        }
        cp_commit();
    };

    float s[DK / 8][4];
    const long long state = (long long)d.dv * DK;
    get_state<DK>(s, W0 ? W0 + b * w0_bs + h * state : nullptr, row0, lane);
    for (int c = 0; c < L::kStages - 1; ++c) issue(c);

    for (int c = 0; c < nch; ++c) {
        cp_wait<L::kStages - 2>();
        __syncthreads();
        issue(c + L::kStages - 1);
        const uint32_t st = sb + (c % L::kStages) * L::stage;
        const uint32_t kt = st, qt = st + L::kK, vt = st + L::kK + L::kQ, gt = vt + L::kV, tm = gt + kGateBytes,
                       am = tm + mat_bytes(P);
        const int left = len - c * CT;

        if (SAVE && (c * CT) % d.gt == 0)
            put_state_parts<DK, P>(s, out.S + ((long long)bh * d.ng + (c * CT) / d.gt) * P * state, d.dv, row0, lane);

        float x[4][4] = {}, z[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
            uint32_t a[P][4];
            as_operand<P>(a, s[2 * kk], s[2 * kk + 1]);
            dot_tokens<DK, P, PK>(x, a, kt, kk, lane);
            if (!SAVE) dot_tokens<DK, P, PK>(z, a, qt, kk, lane);
        }
        // R = V - gamma (W K^T)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float2 ga = lds2(gt + (nb * 8 + 2 * t) * 4);
            float v[4];
            if constexpr (PK == 1) {
                if (nb % 2 == 0) {
                    uint32_t r[4];
                    const int mi = lane >> 3, lr = lane & 7;
                    ldsm4t(r, vt + ((nb * 8 + (mi >> 1) * 8 + lr) * L::VP + warp * 16 + (mi & 1) * 8) * 2);
                    x[nb][0] = fmaf(-ga.x, x[nb][0], lo_f(r[0]));
                    x[nb][1] = fmaf(-ga.y, x[nb][1], hi_f(r[0]));
                    x[nb][2] = fmaf(-ga.x, x[nb][2], lo_f(r[1]));
                    x[nb][3] = fmaf(-ga.y, x[nb][3], hi_f(r[1]));
                    const float2 gb = lds2(gt + (nb * 8 + 8 + 2 * t) * 4);
                    x[nb + 1][0] = fmaf(-gb.x, x[nb + 1][0], lo_f(r[2]));
                    x[nb + 1][1] = fmaf(-gb.y, x[nb + 1][1], hi_f(r[2]));
                    x[nb + 1][2] = fmaf(-gb.x, x[nb + 1][2], lo_f(r[3]));
                    x[nb + 1][3] = fmaf(-gb.y, x[nb + 1][3], hi_f(r[3]));
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = lds1(vt + ((nb * 8 + 2 * t + (q & 1)) * L::VP + warp * 16 + g + (q >> 1) * 8) * 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) x[nb][q] = fmaf(-((q & 1) ? ga.y : ga.x), x[nb][q], v[q]);
            }
        }
        // E = T' R
        float e[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t a[P][4];
            as_operand<P>(a, x[2 * kk], x[2 * kk + 1]);
            mat_nt<P>(e, a, tm, kk, lane);
        }
        if constexpr (SAVE)
            put_rows_parts<P>(wout, e, out.E + ((long long)bh * d.N + (long long)c * CT) * d.dv + row0, out.e_ps, d.dv, left, lane);
        // U = beta E, then gamma_C W + (suffix U)^T K
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float2 be = lds2(gt + (2 * CT + nb * 8 + 2 * t) * 4);
            e[nb][0] *= be.x; e[nb][1] *= be.y; e[nb][2] *= be.x; e[nb][3] *= be.y;
            if (!SAVE) {
                const float2 ga = lds2(gt + (nb * 8 + 2 * t) * 4);
                z[nb][0] *= d.scale * ga.x; z[nb][1] *= d.scale * ga.y; z[nb][2] *= d.scale * ga.x; z[nb][3] *= d.scale * ga.y;
            }
        }
        if (!SAVE) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t a[P][4];
                as_operand<P>(a, e[2 * kk], e[2 * kk + 1]);
                mat_nt<P>(z, a, am, kk, lane);
            }
        }
        const float gc = lds1(gt + (CT - 1) * 4);
#pragma unroll
        for (int nb = 0; nb < DK / 8; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) s[nb][q] *= gc;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float2 su = lds2(gt + (CT + nb * 8 + 2 * t) * 4);
            e[nb][0] *= su.x; e[nb][1] *= su.y; e[nb][2] *= su.x; e[nb][3] *= su.y;
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t a[P][4];
            as_operand<P>(a, e[2 * kk], e[2 * kk + 1]);
            add_outer<DK, P, PK>(s, a, kt, kk, lane);
        }
        if (!SAVE)
            put_tokens<PK>(wout, z, out.Z.p, b * out.Z.bs + h * out.Z.hs + (long long)c * CT * out.Z.ts + row0, out.Z.ts, left, lane);
    }
    cp_wait<0>();
    if (out.W1) put_state<DK>(s, out.W1 + (long long)bh * state, row0, lane);
}

#include "delta_backward.cuh"

// --------------------------------------------------------------------------------------------------
// Workspace
// --------------------------------------------------------------------------------------------------
struct Layout {
    size_t rec, qp, kp, op, E, Y, S, D, dw, total;
};
static Layout layout(const Dims& d, bool fp32, bool backward) {
    const int P = fp32 ? 3 : 2;
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at = align_up(at + bytes, 256); return o; };
    const size_t heads = (size_t)d.B * d.h, toks = heads * d.N;
    l.rec = take(heads * d.nc * rec_bytes(P, backward));
    if (fp32) {
        l.qp = take((size_t)3 * d.B * d.hk * d.N * d.dk * 2);
        l.kp = take((size_t)3 * d.B * d.hk * d.N * d.dk * 2);
    }
    if (backward) {
        if (fp32) l.op = take((size_t)3 * toks * d.dv * 2);
        l.E = take(P * toks * d.dv * 2);
        l.Y = take(P * toks * d.dv * 2);
        l.S = take(heads * d.ng * P * d.dv * d.dk * 2);
        l.D = take(heads * d.ng * P * d.dv * d.dk * 2);
        l.dw = take(heads * d.dv * d.dk * 4);
    }
    l.total = at;
    return l;
}
size_t forward_ws_bytes(const Dims& d, bool fp32) { return layout(d, fp32, false).total; }
size_t backward_ws_bytes(const Dims& d, bool fp32) { return layout(d, fp32, true).total; }

// --------------------------------------------------------------------------------------------------
// Launches
// --------------------------------------------------------------------------------------------------
template <class F>
static cudaError_t allow_smem(F* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// The tokens of x as bf16 parts: x itself (bf16), or 3 parts in the workspace (fp32).
static Parts as_parts(const View& x, bool fp32, uint8_t* ws, const Dims& d, int heads, int width, cudaStream_t st) {
    if (!fp32) return Parts{reinterpret_cast<const __nv_bfloat16*>(x.p), 0, x.bs, x.hs, x.ts};
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(ws);
    const long long n = (long long)d.B * heads * d.N * width;
    const long long blocks = std::min<long long>((n / 4 + 255) / 256, 148 * 16);
    split_tokens<3><<<(unsigned)blocks, 256, 0, st>>>(x, o, n, heads, d.N, width, n / 4);
    return Parts{o, n, (long long)heads * d.N * width, (long long)d.N * width, width};
}

template <int DK, int P, int PK, bool BACKWARD>
static ttt_status run_prep(const Call& c, const Parts& Q, const Parts& K, uint8_t* rec) {
    constexpr int kPrepWarps = prep_warps<DK, PK>(), smem = kPrepWarps * prep_warp_bytes<DK, PK>();
    auto* k = delta_prep<DK, P, PK, BACKWARD>;
    ttt_status st = check_launch(allow_smem(k, smem));
    if (st != TTT_OK) return st;
    const long long total = (long long)c.d.B * c.d.h * c.d.nc;
    k<<<(unsigned)((total + kPrepWarps - 1) / kPrepWarps), kPrepWarps * 32, smem, c.stream>>>(c.d, Q, K, c.G, c.Beta, rec, total);
    return check_launch(cudaGetLastError());
}

template <int DK, int P, int PK, bool SAVE>
static ttt_status run_chain(const Call& c, const Parts& Q, const Parts& K, const uint8_t* rec, const ChainOut& out) {
    constexpr int NW = 4;
    using L = ChainLayout<DK, P, PK, NW, SAVE>;
    static_assert(L::smem <= 227 * 1024, "shared memory of a chain CTA");
    auto* k = delta_chain<DK, P, PK, NW, SAVE>;
    ttt_status st = check_launch(allow_smem(k, L::smem));
    if (st != TTT_OK) return st;
    k<<<(unsigned)(c.d.B * c.d.h * (c.d.dv / L::VW)), NW * 32, L::smem, c.stream>>>(c.d, Q, K, c.V, rec, c.W0, c.w0_bs, out);
    return check_launch(cudaGetLastError());
}

template <int DK, int P, int PK>
static ttt_status forward_t(const Call& c) {
    const Layout l = layout(c.d, PK == 3, false);
    const Parts Q = as_parts(c.Q, PK == 3, c.ws + l.qp, c.d, c.d.hk, DK, c.stream);
    const Parts K = as_parts(c.K, PK == 3, c.ws + l.kp, c.d, c.d.hk, DK, c.stream);
    ttt_status st = run_prep<DK, P, PK, false>(c, Q, K, c.ws + l.rec);
    if (st != TTT_OK) return st;
    ChainOut out{};
    out.Z = c.Z;
    out.W1 = c.W1_out;
    return run_chain<DK, P, PK, false>(c, Q, K, c.ws + l.rec, out);
}

template <int DK, int P, int PK>
static ttt_status backward_t(const Call& c) {
    constexpr bool F = PK == 3;
    const Layout l = layout(c.d, F, true);
    const Parts Q = as_parts(c.Q, F, c.ws + l.qp, c.d, c.d.hk, DK, c.stream);
    const Parts K = as_parts(c.K, F, c.ws + l.kp, c.d, c.d.hk, DK, c.stream);
    const Parts O = as_parts(c.Z, F, c.ws + l.op, c.d, c.d.h, c.d.dv, c.stream);
    uint8_t* rec = c.ws + l.rec;
    ttt_status st = run_prep<DK, P, PK, true>(c, Q, K, rec);
    if (st != TTT_OK) return st;
    const long long ps = (long long)c.d.B * c.d.h * c.d.N * c.d.dv;
    ChainOut out{};
    out.E = reinterpret_cast<__nv_bfloat16*>(c.ws + l.E);
    out.e_ps = ps;
    out.S = reinterpret_cast<__nv_bfloat16*>(c.ws + l.S);
    st = run_chain<DK, P, PK, true>(c, Q, K, rec, out);
    if (st != TTT_OK) return st;
    BackOut bo{};
    bo.dV = c.dV;
    bo.Y = reinterpret_cast<__nv_bfloat16*>(c.ws + l.Y);
    bo.y_ps = ps;
    bo.D = reinterpret_cast<__nv_bfloat16*>(c.ws + l.D);
    const bool reduce = c.dW0 && c.w0_bs == 0;
    bo.dW0 = reduce ? reinterpret_cast<float*>(c.ws + l.dw) : c.dW0;
    st = run_reverse<DK, P, PK>(c, Q, K, O, rec, bo);
    if (st != TTT_OK) return st;
    st = run_grads<DK, P, PK>(c, Q, K, O, out, bo);
    if (st != TTT_OK || !reduce) return st;
    return run_sum_images(bo.dW0, c.dW0, c.d.B, (long long)c.d.h * c.d.dv * DK, c.stream);
}

ttt_status launch_forward(const Call& c) {
    if (c.fp32) return c.d.dk == 64 ? forward_t<64, 3, 3>(c) : forward_t<128, 3, 3>(c);
    return c.d.dk == 64 ? forward_t<64, 2, 1>(c) : forward_t<128, 2, 1>(c);
}
ttt_status launch_backward(const Call& c) {
    if (c.fp32) return c.d.dk == 64 ? backward_t<64, 3, 3>(c) : backward_t<128, 3, 3>(c);
    return c.d.dk == 64 ? backward_t<64, 2, 1>(c) : backward_t<128, 2, 1>(c);
}

}  // namespace gd
}  // namespace ttt
