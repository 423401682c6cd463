// delta_tc.cuh -- the sequential part of the gated delta rule for bf16 tokens, on tcgen05 (included by delta.cu,
// inside ttt::gd; the formulas are in delta.cu and delta_backward.cuh).
//
// One CTA per value head (and image): its d_v rows of the state are lanes of tensor memory, where the fp32 state
// stays for the whole sequence.  Chunks of 64 tokens.  In the products the left operand is always a [d_v x .] matrix in
// tensor memory as two bf16 parts, written there by the eight chain warps; the right operands are token
// tiles and the chunk's 64 x 64 matrices in shared memory, brought by TMA as they are.  Per chunk (forward):
//   state -> parts | X = W K^T | R = V - gamma X -> parts | E = T' R | U = beta E, suffix U -> parts | W = gamma_C W + U^T K
// with Q W^T and A U for the readout issued where the tensor core would wait, and read out by four warps
// of their own.
//
// d_v = 64: products of 64 rows, whose accumulators use 16 of each 32 lanes.
//
// Bound: the chain of a chunk, about 5,500 cycles at d = 128: 36 products of 45 cycles one after another and, between
// them, four elementwise passes over [d_v x 64 .. d_k] values by eight warps.  In the adjoint's sweep (9,000 cycles) the four
// output warps, which write the adjoint's and Y's parts and dV.  148 heads of 2048 tokens, d = 128: forward 230 us,
// backward 796 us.

constexpr int TC = 64;                        // tokens per chunk
constexpr int MV = 128;                       // rows of the state, d_v: the lanes of tensor memory
constexpr int kTcGates = 1024;                // gamma, suffix, beta (3 x 64 fp32), padded
constexpr int kTcMat = 2 * TC * 128;          // two parts of a 64 x 64 bf16 matrix, rows of 128 swizzled bytes
__host__ __device__ constexpr int tc_rec_bytes(bool backward) { return kTcGates + (backward ? 3 : 2) * kTcMat; }

// One thread of a converged warp.  Products issued inside `if (elect_one())` from warp-uniform descriptors take the
// tensor core's own time (35 cycles for 128 x 64 x 16); behind `lane == 0` the compiler moves every operand
// to a uniform register first (about 50).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
    return e != 0;
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t col, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 16) tmem_ld16(col + i, *reinterpret_cast<float(*)[16]>(&v[i]));
    tmem_ld_wait();
}
// D (tensor memory) += A (tensor memory, bf16 pairs) * B (shared memory)
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d_at(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2, int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(m), "r"(s32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// --------------------------------------------------------------------------------------------------
// Prep: the 64 x 64 matrices.  One CTA of four warps per chunk.  The inverses start from the four 16 x 16 blocks on the
// diagonal (forward substitution, one warp each) and are joined pair by pair on matrix instructions: with 32 x 32 blocks and
// fp32 products the kernel took a third longer (forward, 148 heads of 2048 tokens: 271 us against 230 in all).
// --------------------------------------------------------------------------------------------------
constexpr int GP2 = TC + 4;                   // row pitch (floats) of the 64 x 64 matrices

template <int DK, bool BACKWARD>
struct Prep64 {
    static constexpr int KP = DK + 8, mat = TC * GP2 * 4;
    static constexpr int tiles = 2 * TC * KP * 2;
    static constexpr int front = tiles > 2 * mat ? tiles : 2 * mat;                // K and Q tiles, then G and Q K^T, then G and T'
    static constexpr int oU = (front + 127) / 128 * 128, oImg = oU + (BACKWARD ? mat : 0);   // T_u; one image at a time
    static constexpr int oRow = oImg + kTcMat;                 // g, beta, suffix inside 16
    static constexpr int smem = oRow + 3 * TC * 4;
};

// Elements (i, j) and (i, j + 1), j even, of a two-part 64 x 64 image.
__device__ __forceinline__ void put_pair(uint8_t* img, int i, int j, float x, float y) {
    uint32_t w[2];
    split2<2>(x, y, w);
    uint8_t* o = img + i * 128 + (((j >> 3) ^ (i & 7)) << 4) + (j & 7) * 2;
    *reinterpret_cast<uint32_t*>(o) = w[0];
    *reinterpret_cast<uint32_t*>(o + TC * 128) = w[1];
}

// Inverses of I + L, L = G diag(beta) (T', lanes 0-15) and diag(beta) G (T_u, lanes 16-31), for a 16 x 16 diagonal block
// of G: a column per lane, by forward substitution.
__device__ __forceinline__ void solve16(const float* g, const float* beta, float* out, int lane) {
    const bool u = lane >= 16;
    const int col = lane & 15;
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int l = 0; l < 16; l += 4) {
            if (l >= i) continue;
            const float4 v = *reinterpret_cast<const float4*>(g + i * GP2 + l);
            s[0] = fmaf(v.x, y[l], s[0]);
            if (l + 1 < i) s[1] = fmaf(v.y, y[l + 1], s[1]);
            if (l + 2 < i) s[2] = fmaf(v.z, y[l + 2], s[2]);
            if (l + 3 < i) s[3] = fmaf(v.w, y[l + 3], s[3]);
        }
        const float be = beta[i], sum = (s[0] + s[1]) + (s[2] + s[3]);
        const float x = (i == col ? 1.f : 0.f) - (u ? be * sum : sum);
        if (out) out[i * GP2 + col] = i >= col ? x : 0.f;
        y[i] = u ? x : be * x;
    }
}
// The block below two inverted diagonal blocks of 16 KS: acc = T_22 L_21 T_11, rows 16 strip .., columns col0 .. col0 + 15
// (U: of T_u, else of T').  The first product's accumulators are the second one's left operand.  Operands as two
// bf16 parts, the product of the low ones dropped: about 16 bits, as the inverse is handed on.
template <int KS, bool U>
__device__ __forceinline__ void below(float (&acc)[2][4], const float* g21, const float* beta1, const float* beta2, const float* t22,
                                      const float* t11, int strip, int col0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t m[KS][2][4];                          // T_22 L_21 as parts, [16 columns][part]
    {
        float c[2 * KS][4] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks > strip) continue;              // T_22 is lower triangular
            uint32_t a[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = *reinterpret_cast<const float2*>(t22 + (strip * 16 + g + (e & 1) * 8) * GP2 + ks * 16 + 2 * t + (e >> 1) * 8);
                uint32_t w[2];
                split2<2>(v.x, v.y, w);
                a[0][e] = w[0];
                a[1][e] = w[1];
            }
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n) {
                uint32_t b[2][2];
                const float right = U ? 1.f : beta1[n * 8 + g];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = ks * 16 + 2 * t + e * 8;
                    const float2 left = U ? *reinterpret_cast<const float2*>(beta2 + k) : make_float2(right, right);
                    uint32_t w[2];
                    split2<2>(left.x * g21[k * GP2 + n * 8 + g], left.y * g21[(k + 1) * GP2 + n * 8 + g], w);
                    b[0][e] = w[0];
                    b[1][e] = w[1];
                }
                mma16816(c[n], a[0], b[0][0], b[0][1]);
                mma16816(c[n], a[0], b[1][0], b[1][1]);
                mma16816(c[n], a[1], b[0][0], b[0][1]);
            }
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w[2];
                split2<2>(c[2 * ks + (e >> 1)][(e & 1) * 2], c[2 * ks + (e >> 1)][(e & 1) * 2 + 1], w);
                m[ks][0][e] = w[0];
                m[ks][1][e] = w[1];
            }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t b[2][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float* x = t11 + (ks * 16 + 2 * t + e * 8) * GP2 + col0 + n * 8 + g;
                uint32_t w[2];
                split2<2>(x[0], x[GP2], w);
                b[0][e] = w[0];
                b[1][e] = w[1];
            }
            mma16816(acc[n], m[ks][0], b[0][0], b[0][1]);
            mma16816(acc[n], m[ks][0], b[1][0], b[1][1]);
            mma16816(acc[n], m[ks][1], b[0][0], b[0][1]);
        }
    }
}
// Joins the four 16 x 16 blocks on the diagonal of a 64 x 64 inverse at t (fp32, zeros above) pair by pair ..
template <bool U>
__device__ __forceinline__ void join16(const float* gm, const float* beta, float* t, int pair, int lane) {
    const int o = pair * 32;
    float acc[2][4];
    below<1, U>(acc, gm + (o + 16) * GP2 + o, beta + o, beta + o + 16, t + (o + 16) * GP2 + o + 16, t + o * GP2 + o, 0, 0, lane);
    float* x = t + (o + 16 + (lane >> 2)) * GP2 + o + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        *reinterpret_cast<float2*>(x + n * 8) = make_float2(-acc[n][0], -acc[n][1]);
        *reinterpret_cast<float2*>(x + n * 8 + 8 * GP2) = make_float2(-acc[n][2], -acc[n][3]);
    }
}
// .. and writes the whole inverse, its last block among it, as an image.
template <bool U>
__device__ __forceinline__ void join32(const float* gm, const float* beta, const float* t, uint8_t* img, int warp, int lane) {
    const int strip = warp >> 1, col0 = (warp & 1) * 16;
    float acc[2][4];
    below<2, U>(acc, gm + 32 * GP2, beta, beta + 32, t + 32 * GP2 + 32, t, strip, col0, lane);
    const int i = 32 + strip * 16 + (lane >> 2), j = col0 + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        put_pair(img, i, j + n * 8, -acc[n][0], -acc[n][1]);
        put_pair(img, i + 8, j + n * 8, -acc[n][2], -acc[n][3]);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int x = warp * 16 + r * 2 + (lane >> 4), y = (x & 32) + (lane & 15) * 2;
        const float2 v = *reinterpret_cast<const float2*>(t + x * GP2 + y);
        put_pair(img, x, y, v.x, v.y);
    }
}

template <int DK, bool BACKWARD>
__global__ void __launch_bounds__(128)
delta_prep64(Dims d, Parts Q, Parts K, View G, View Beta, uint8_t* rec, uint32_t* err) {
    using L = Prep64<DK, BACKWARD>;
    constexpr int KP = L::KP;
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0 && tid == 0) *err = 0;
    const int nc = (d.N + TC - 1) / TC;
    const int c = blockIdx.x % nc, bh = blockIdx.x / nc, h = bh % d.h, b = bh / d.h;
    const int left = seq_len(d, b) - c * TC;
    if (left <= 0) return;
    const uint32_t kt = s32(smem), qt = kt + TC * KP * 2;
    float* kkm = reinterpret_cast<float*>(smem);
    float* qkm = kkm + TC * GP2;
    float* tm = qkm;                                           // T', once Q K^T is used up
    float* um = reinterpret_cast<float*>(smem + L::oU);
    uint8_t* img = smem + L::oImg;
    float* gr = reinterpret_cast<float*>(smem + L::oRow);
    float *br = gr + TC, *s16 = br + TC;
    {
        const char* ks = reinterpret_cast<const char*>(K.p + b * K.bs + (h / d.r) * K.hs + (long long)c * TC * K.ts);
        const char* qs = reinterpret_cast<const char*>(Q.p + b * Q.bs + (h / d.r) * Q.hs + (long long)c * TC * Q.ts);
        constexpr int CPR = DK / 8, RPI = 128 / CPR;
        const int r0 = tid / CPR, col = tid % CPR;
#pragma unroll 4
        for (int r = r0; r < TC; r += RPI) {
            const bool live = r < left;
            const long long o = live ? r : 0;
            cp16(kt + (r * KP + col * 8) * 2, ks + o * K.ts * 2 + col * 16, live);
            cp16(qt + (r * KP + col * 8) * 2, qs + o * Q.ts * 2 + col * 16, live);
        }
        cp_commit();
    }
    uint8_t* out = rec + (long long)blockIdx.x * tc_rec_bytes(BACKWARD);
    if (warp < 2) {                                            // gates of tokens 32 warp + lane; none behind the sequence's end
        const int t = warp * 32 + lane;
        const bool live = t < left;
        const long long tok = (long long)c * TC + t;
        const float g = live ? reinterpret_cast<const float*>(G.p)[b * G.bs + h * G.hs + tok * G.ts] : 0.f;
        const float beta = live ? reinterpret_cast<const float*>(Beta.p)[b * Beta.bs + h * Beta.hs + tok * Beta.ts] : 0.f;
        const int l16 = lane & 15;
        float pre = g, suf = __shfl_down_sync(~0u, g, 1, 16);
        if (l16 == 15) suf = 0.f;
#pragma unroll
        for (int o = 1; o < 16; o *= 2) {
            const float a = __shfl_up_sync(~0u, pre, o, 16), z = __shfl_down_sync(~0u, suf, o, 16);
            if (l16 >= o) pre += a;
            if (l16 + o < 16) suf += z;
        }
        gr[t] = g;
        br[t] = beta;
        s16[t] = suf;
        asm volatile("bar.sync 1, 64;" ::: "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q) {                          // the other sixteens' sums
            const float all = gr[q * 16] + s16[q * 16];
            if (q < t / 16) pre += all;
            if (q > t / 16) suf += all;
        }
        float* gates = reinterpret_cast<float*>(out);
        gates[t] = expf(pre);
        gates[TC + t] = expf(suf);
        gates[2 * TC + t] = beta;
    }
    for (int x = tid; x < kTcMat / 16; x += 128) reinterpret_cast<uint4*>(img)[x] = make_uint4(0, 0, 0, 0);   // what lies above the diagonal
    auto copy_out = [&](int m) {
#pragma unroll
        for (int x = 0; x < kTcMat / 16; x += 128)
            reinterpret_cast<uint4*>(out + kTcGates + m * kTcMat)[x + tid] = reinterpret_cast<const uint4*>(img)[x + tid];
    };
    cp_wait<0>();
    __syncthreads();
    {
        // K K^T rows 16 w .. and Q K^T rows 16 (3 - w) ..: ten 16 x 8 blocks on or below the diagonal per warp
        float m[2][8][4] = {};
        const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
            uint32_t a0[4], a1[4];
            const uint32_t ao = ((((mi & 1) * 8 + lr)) * KP + kk * 16 + (mi >> 1) * 8) * 2;
            ldsm4(a0, kt + ao + warp * 16 * KP * 2);
            ldsm4(a1, qt + ao + (3 - warp) * 16 * KP * 2);
#pragma unroll
            for (int n2 = 0; n2 < 4; ++n2) {
                if (n2 > max(warp, 3 - warp)) continue;
                uint32_t w[4];
                ldsm4(w, kt + ((n2 * 16 + (mi >> 1) * 8 + lr) * KP + kk * 16 + (mi & 1) * 8) * 2);
                if (n2 <= warp) {
                    mma16816(m[0][2 * n2], a0, w[0], w[1]);
                    mma16816(m[0][2 * n2 + 1], a0, w[2], w[3]);
                }
                if (n2 <= 3 - warp) {
                    mma16816(m[1][2 * n2], a1, w[0], w[1]);
                    mma16816(m[1][2 * n2 + 1], a1, w[2], w[3]);
                }
            }
        }
        __syncthreads();                                       // the tiles have been read
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int block = e ? 3 - warp : warp;
            float* o = (e ? qkm : kkm) + (block * 16 + g) * GP2 + 2 * t;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n > 2 * block + 1) continue;
                *reinterpret_cast<float2*>(o + n * 8) = make_float2(m[e][n][0], m[e][n][1]);
                *reinterpret_cast<float2*>(o + 8 * GP2 + n * 8) = make_float2(m[e][n][2], m[e][n][3]);
            }
        }
    }
    __syncthreads();
    {
        // Gamma: warp w takes rows 16 w .. 16 w + 15, a lane two columns; logs summed from zero at i = j
        const int j = 2 * lane, jb = lane >> 3;
        float s0 = 0.f, s1 = 0.f;
        if (jb < warp) {
            s0 = s16[j];
            s1 = s16[j + 1];
            for (int q = jb + 1; q < warp; ++q) {
                const float all = gr[q * 16] + s16[q * 16];
                s0 += all;
                s1 += all;
            }
        }
        if (jb <= warp) {
#pragma unroll 4
            for (int i = warp * 16; i < warp * 16 + 16; ++i) {
                const float gi = gr[i];
                if (i > j) s0 += gi;
                if (i > j + 1) s1 += gi;
                const float d0 = i >= j ? __expf(s0) : 0.f, d1 = i > j ? __expf(s1) : 0.f;      // relative error about 2^-22 (1 + |s|)
                float2* kk = reinterpret_cast<float2*>(kkm + i * GP2 + j);
                const float2 a = *reinterpret_cast<const float2*>(qkm + i * GP2 + j), x = *kk;
                put_pair(img, i, j, i >= j ? d.scale * d0 * a.x : 0.f, i > j ? d.scale * d1 * a.y : 0.f);
                *kk = make_float2(i > j ? d0 * x.x : 0.f, i > j + 1 ? d1 * x.y : 0.f);
            }
        }
    }
    __syncthreads();
    copy_out(1);                                               // A
    {
        const int o = warp * 16;
        float* dst = lane < 16 ? tm : BACKWARD ? um : nullptr;
        solve16(kkm + o * GP2 + o, br + o, dst ? dst + o * GP2 + o : nullptr, lane);
        if (!(warp & 1) && dst)                                // right of it, above the diagonal
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[(o + i) * GP2 + o + 16 + (lane & 15)] = 0.f;
    }
    __syncthreads();
    if (warp < 2) join16<false>(kkm, br, tm, warp, lane);
    if (BACKWARD && warp >= 2) join16<true>(kkm, br, um, warp - 2, lane);
    __syncthreads();
    join32<false>(kkm, br, tm, img, warp, lane);
    __syncthreads();
    copy_out(0);
    if constexpr (BACKWARD) {
        __syncthreads();
        join32<true>(kkm, br, um, img, warp, lane);
        __syncthreads();
        copy_out(2);
    }
}

// --------------------------------------------------------------------------------------------------
// Chain
// --------------------------------------------------------------------------------------------------
// A bf16 token tensor: boxes of 64 tokens x 64 features (swizzled), and the plain view behind it.
struct Tok64 {
    CUtensorMap map;
    const __nv_bfloat16* p;
    long long bs, hs, ts;
    int hmul, bmul;
};
// Loads features [0, W) of 64 tokens into [W / 64][64 tokens][128 bytes].  Whole chunks come by TMA (the return value: bytes
// to expect); of a partial one the warp copies the rows itself, the last token's row standing for those past the end.
template <int W>
__device__ __forceinline__ uint32_t tok64_bytes(int left) { return left >= TC ? W * 128 : 0; }
template <int W>
__device__ __forceinline__ void tok64_tail(uint32_t dst, const Tok64& x, int b, int head, int tok, int left, int lane) {
    constexpr int CPR = W / 8;
    const __nv_bfloat16* src = x.p + b * x.bs + head * x.hs + (long long)tok * x.ts;
    for (int i = lane; i < TC * CPR; i += 32) {
        const int row = i / CPR, pc = i % CPR;
        const uint4 v = *reinterpret_cast<const uint4*>(src + min(row, left - 1) * x.ts + pc * 8);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (pc >> 3) * TC * 128 + row * 128 + (((pc & 7) ^ (row & 7)) << 4)),
                     "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
    }
}
template <int W>
__device__ __forceinline__ void tok64_load(uint32_t dst, const Tok64& x, uint64_t* bar, int b, int head, int tok) {
#pragma unroll
    for (int c = 0; c < W / 64; ++c) tma_load_5d_at(dst + c * TC * 128, &x.map, bar, c * 64, tok, head * x.hmul, b * x.bmul, 0);
}
__device__ __forceinline__ void bulk_at(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(s32(bar))
                 : "memory");
}

struct TcArgs {
    Dims d;
    Tok64 K, Q, V;                     // V: values (forward) or dZ (reverse)
    const uint8_t* rec;
    int rec_bytes;
    const float* W0;                   // start (forward) or dW1 (reverse), nullable
    long long w0_bs;
    float* W1;                         // nullable: last state, or the gradient of the first, [B][h][dv][dk]
    View Z;                            // forward: the readout; reverse: dV
    CUtensorMap mZ, mE, mS;            // Z; E (or Y) [2][B][h][N][dv]; states (adjoints) at the chunks' starts (ends) [B][h][ng][2][dv][dk]
    int zh, zb;                        // 0 where Z has one head or image
    uint32_t* err;
    unsigned long long wait_ns;
};

struct TcCtl {
    uint64_t full[3], empty[3], sp, xd, rp, ed, up, sd, z1, z1free, z2, z2free, spfree, fr, spa, ur;
    uint32_t tmem;
    int abort_flag;
};

// acc [. x 64 tokens] = (the state's parts) X^T, X a token tile, issued by one thread of the calling warp.  d_k = 128: in
// two halves, the first 32 columns of each warp half's 64, then the others, as the chain warps write them.
template <int DK>
__device__ __forceinline__ void state_product(uint32_t acc, uint32_t parts, uint32_t x, uint32_t id, int half) {
    if (elect_one()) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kk = DK == 128 ? (i / 2) * 4 + half * 2 + i % 2 : i;
#pragma unroll
            for (int part = 0; part < 2; ++part)
                mma_bf16_ts(acc, parts + part * (DK / 2) + kk * 8, sdesc_sw128(x + (kk / 4) * TC * 128 + (kk % 4) * 32, 16, 1024), id,
                            half > 0 || i > 0 || part > 0);
        }
    }
    __syncwarp();
}

template <int DK, bool SAVE>
struct TcChain {
    static constexpr int oT = kTcGates, oA = oT + kTcMat, oK = oA + (SAVE ? 0 : kTcMat), oQ = oK + DK * 128, oV = oQ + (SAVE ? 0 : DK * 128);
    static constexpr int stage = oV + MV * 128;
    static constexpr int kStages = SAVE ? 3 : 2, kSlots = SAVE ? 3 : 2;
    static constexpr int used = kStages * stage + kSlots * MV * 128 + 512 + 1024, smem = used > 116 * 1024 ? used : 116 * 1024;   // one CTA per SM
    static_assert(smem <= 227 * 1024 && stage % 1024 == 0, "shared memory of a chain CTA");
    // tensor-memory columns: state, its parts (hi, lo), X / E / A U, R then U parts, suffix U parts, Q W^T
    static constexpr uint32_t cS = 0, cP = DK, cX = 2 * DK, cR = cX + 64, cU = cR + 64, cZ = cU + 64;
};

// Packed bf16 parts of 32 values -> 16 tensor-memory columns at `hi` and 16 at `lo`.
__device__ __forceinline__ void tmem_st_parts(uint32_t hi, uint32_t lo, const float (&v)[32]) {
    uint32_t h[16], l[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        h[i] = pack2(v[2 * i], v[2 * i + 1]);
        const float2 rest = ffma2(make_float2(lo_f(h[i]), hi_f(h[i])), make_float2(-1.f, -1.f), make_float2(v[2 * i], v[2 * i + 1]));
        l[i] = pack2(rest.x, rest.y);
    }
    tmem_st16(hi, h);
    tmem_st16(lo, l);
}
// Releases what a warp wrote to tensor memory (or has read from it) to whoever waits on `bar`.
__device__ __forceinline__ void tc_arrive(uint64_t* bar, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
// The four output warps' way to global memory: tiles are laid out in a ring of shared-memory slots as TMA reads
// them (rows of 128 bytes, swizzled) and stored by it; one thread issues the stores.
template <int SLOTS>
struct OutRing {
    static constexpr int kSlot = MV * 128;
    uint32_t base;
    int lane;
    bool issuer;
    int job;
    __device__ __forceinline__ uint32_t open() {       // a slot that no store still reads
        if (issuer) bulk_wait_read<SLOTS - 1>();
        named_bar_sync(3, 128);
        return base + (job++ % SLOTS) * kSlot;
    }
    __device__ __forceinline__ void ready() {
        fence_proxy_async_smem();
        named_bar_sync(3, 128);
    }
    __device__ __forceinline__ void store(const CUtensorMap* m, uint32_t slot, int c0, int c1, int c2, int c3) {
        asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5, 0}], [%1];" ::"l"(m), "r"(slot), "r"(c0),
                     "r"(c1), "r"(c2), "r"(c3)
                     : "memory");
    }
    // this thread's row of a [MV][64] tile: 32 packed pairs
    __device__ __forceinline__ void put_row(uint32_t slot, int row, const float (&v)[32]) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(slot + row * 128 + ((k ^ (row & 7)) << 4)), "f"(v[4 * k]), "f"(v[4 * k + 1]),
                         "f"(v[4 * k + 2]), "f"(v[4 * k + 3])
                         : "memory");
    }
    // this thread's feature of 32 tokens from t0 on of a [MV / 64][64 tokens][64] tile, rounded to bf16
    __device__ __forceinline__ void put_column(uint32_t slot, int row, int t0, const float (&v)[32]) {
        const uint32_t at = slot + (row >> 6) * TC * 128 + t0 * 128 + (row & 7) * 2, pc = (row & 63) >> 3;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const uint32_t w = pack2(v[i], v[i + 1]);
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(at + i * 128 + ((pc ^ (i & 7)) << 4)), "h"((uint16_t)w) : "memory");
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(at + (i + 1) * 128 + ((pc ^ ((i + 1) & 7)) << 4)), "h"((uint16_t)(w >> 16)) : "memory");
        }
    }
    // Rows [0, left) of a token tile to a strided tensor: by TMA where the chunk is whole, else by the warps themselves.
    __device__ __forceinline__ void tokens_out(const CUtensorMap* m, uint32_t slot, __nv_bfloat16* dst, long long ts, int tok, int head, int img,
                                               int left, int tid) {
        if (left >= TC) {
            if (issuer) {
#pragma unroll
                for (int c = 0; c < MV / 64; ++c) store(m, slot + c * TC * 128, c * 64, tok, head, img);
                bulk_commit();
            }
            return;
        }
        if (issuer) bulk_commit();                     // an empty group: jobs and groups stay in step
        for (int x = tid; x < left * (MV / 8); x += 128) {
            const int r = x / (MV / 8), pc = x % (MV / 8);
            const uint4 v = lds4u(slot + (pc >> 3) * TC * 128 + r * 128 + (((pc & 7) ^ (r & 7)) << 4));
            *reinterpret_cast<uint4*>(dst + r * ts + pc * 8) = v;
        }
    }
};

template <int DK, bool SAVE>
__device__ __forceinline__ void chain_tc_body(const TcArgs& p, int bh) {
    using L = TcChain<DK, SAVE>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (s32(smem_raw) & 1023));
    const uint32_t sb = s32(smem);
    TcCtl& ctl = *reinterpret_cast<TcCtl*>(smem + L::kStages * L::stage + L::kSlots * MV * 128);
    const Dims& d = p.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = bh / d.h, h = bh % d.h;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int len = seq_len(d, b), nch = (len + TC - 1) / TC;
    const long long state = (long long)d.dv * DK;
    const Abort ab{&ctl.abort_flag, p.err, p.wait_ns};
    if (tid == 0) {
        ctl.abort_flag = 0;
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 13);
        }
        for (uint64_t* x : {&ctl.xd, &ctl.ed, &ctl.sd, &ctl.z1, &ctl.z2}) mbar_init(x, 1);
        for (uint64_t* x : {&ctl.spa, &ctl.sp, &ctl.rp, &ctl.up, &ctl.ur}) mbar_init(x, 8);
        for (uint64_t* x : {&ctl.z1free, &ctl.z2free, &ctl.spfree}) mbar_init(x, 4);
        fence_barrier_init();
    }
    if (warp == 13) {
        tmem_alloc(&ctl.tmem, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tm = 0;                     // all 512 columns are this CTA's: they start at 0
    auto full_wait = [&](int c) { return mbar_wait(&ctl.full[c % L::kStages], (c / L::kStages) & 1, ab); };

    if (warp == 12) {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        int c = 0;
        for (; c < nch; ++c) {
            const int s = c % L::kStages, left = len - c * TC;
            if (c >= L::kStages) ok = mbar_wait(&ctl.empty[s], (c / L::kStages - 1) & 1, ab);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            const uint32_t st = sb + s * L::stage;
            if (left < TC) {
                tok64_tail<DK>(st + L::oK, p.K, b, h / d.r, c * TC, left, lane);
                if (!SAVE) tok64_tail<DK>(st + L::oQ, p.Q, b, h / d.r, c * TC, left, lane);
                tok64_tail<MV>(st + L::oV, p.V, b, h, c * TC, left, lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) {
                constexpr uint32_t rb = kTcGates + (SAVE ? 1 : 2) * kTcMat;
                mbar_arrive_expect_tx(&ctl.full[s], rb + tok64_bytes<DK>(left) * (SAVE ? 1 : 2) + tok64_bytes<MV>(left));
                bulk_at(st, p.rec + ((long long)bh * d.nc + c) * p.rec_bytes, rb, &ctl.full[s]);
                if (left >= TC) {
                    tok64_load<DK>(st + L::oK, p.K, &ctl.full[s], b, h / d.r, c * TC);
                    tok64_load<MV>(st + L::oV, p.V, &ctl.full[s], b, h, c * TC);
                    if (!SAVE) tok64_load<DK>(st + L::oQ, p.Q, &ctl.full[s], b, h / d.r, c * TC);
                }
            }
            __syncwarp();
        }
        // nothing may still be on its way when the CTA ends
        for (int i = max(0, c - L::kStages); i < c; ++i) mbar_drain(&ctl.full[i % L::kStages], (i / L::kStages) & 1, drain_limit(ab));
    } else if (warp == 13) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t id64 = idesc_bf16_f32(MV, 64, false, false), idS = idesc_bf16_f32(MV, DK, false, true);
        bool ok = true;
        int c = 0;
        for (; c < nch; ++c) {
            const uint32_t ph = c & 1, st = sb + (c % L::kStages) * L::stage;
            ok = full_wait(c);
            if (c > 0) ok = ok && mbar_wait(&ctl.z2free, ph ^ 1, ab);          // X's place has been read out
            ok = ok && mbar_wait(&ctl.spa, ph, ab);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            state_product<DK>(tm + L::cX, tm + L::cP, st + L::oK, id64, 0);
            if (DK == 128) {
                ok = __all_sync(~0u, mbar_wait(&ctl.sp, ph, ab));
                if (!ok) break;
                tc_fence_after();
                state_product<DK>(tm + L::cX, tm + L::cP, st + L::oK, id64, 1);
            }
            if (elect_one()) mma_commit(&ctl.xd);
            __syncwarp();
            if (!SAVE) {
                if (c > 0) ok = mbar_wait(&ctl.z1free, ph ^ 1, ab);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                state_product<DK>(tm + L::cZ, tm + L::cP, st + L::oQ, id64, 0);
                if (DK == 128) state_product<DK>(tm + L::cZ, tm + L::cP, st + L::oQ, id64, 1);
                if (elect_one()) mma_commit(&ctl.z1);
                __syncwarp();
            }
            ok = mbar_wait(&ctl.rp, ph, ab);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            // E = T' R: rows of T' (columns of the product) from 16 kk on meet tokens 16 kk .. 16 kk + 15
            auto lower = [&](uint32_t dcol, uint32_t a, uint32_t mat) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t id = kk == 0 ? idesc_bf16_f32(MV, 64, false, false) : kk == 1 ? idesc_bf16_f32(MV, 48, false, false)
                                      : kk == 2 ? idesc_bf16_f32(MV, 32, false, false) : idesc_bf16_f32(MV, 16, false, false);
                    const uint64_t hi = sdesc_sw128(mat + kk * 2048 + kk * 32, 16, 1024), lo = sdesc_sw128(mat + TC * 128 + kk * 2048 + kk * 32, 16, 1024);
                    mma_bf16_ts(dcol + kk * 16, a + kk * 8, hi, id, kk > 0);
                    mma_bf16_ts(dcol + kk * 16, a + kk * 8, lo, id, 1);
                    mma_bf16_ts(dcol + kk * 16, a + 32 + kk * 8, hi, id, 1);
                }
            };
            if (elect_one()) {
                lower(tm + L::cX, tm + L::cR, st + L::oT);
                mma_commit(&ctl.ed);
            }
            __syncwarp();
            ok = mbar_wait(&ctl.up, ph, ab);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        mma_bf16_ts(tm + L::cS, tm + L::cU + part * 32 + kk * 8, sdesc_sw128(st + L::oK + kk * 2048, TC * 128, 1024), idS, 1);
                mma_commit(&ctl.sd);
                if (SAVE) mma_commit(&ctl.empty[c % L::kStages]);
            }
            __syncwarp();
            if (!SAVE) {
                ok = __all_sync(~0u, mbar_wait(&ctl.ur, ph, ab));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    lower(tm + L::cX, tm + L::cR, st + L::oA);                 // A U, over E
                    mma_commit(&ctl.z2);
                    mma_commit(&ctl.empty[c % L::kStages]);
                }
                __syncwarp();
            }
        }
        // the last products end before the CTA gives its tensor memory back
        if (!ok) {
            if (elect_one()) mma_commit(&ctl.sd);
            __syncwarp();
            mbar_drain(&ctl.sd, c & 1, drain_limit(ab));
        } else if (nch > 0) {
            mbar_drain(SAVE ? &ctl.sd : &ctl.z2, (nch - 1) & 1, drain_limit(ab));
        }
    } else {
        // rows of the state: tensor-memory lane <-> row of this thread
        const int q = warp & 3;
        const uint32_t lofs = (uint32_t)(q * 32) << 16;
        const int row = q * 32 + lane;
        bool ok = true;
        if (warp < 8) {
            // ------------------------------------------------------------ chain
            const int hf = warp >> 2, k0 = hf * (DK / 2);              // this warp's half of the columns
            const float* w0 = p.W0 ? p.W0 + b * p.w0_bs + h * state + (long long)row * DK + k0 : nullptr;
#pragma unroll
            for (int k = 0; k < DK / 2; k += 16) {
                uint32_t r[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 v = w0 ? *reinterpret_cast<const float4*>(w0 + k + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    r[i] = __float_as_uint(v.x); r[i + 1] = __float_as_uint(v.y); r[i + 2] = __float_as_uint(v.z); r[i + 3] = __float_as_uint(v.w);
                }
                tmem_st16(tm + L::cS + lofs + k0 + k, r);
            }
            tmem_st_wait();
            for (int c = 0; c < nch; ++c) {
                const uint32_t ph = c & 1;
                const uint8_t* st = smem + (c % L::kStages) * L::stage;
                const float* gam = reinterpret_cast<const float*>(st);
                ok = full_wait(c);
                if (c > 0) ok = ok && mbar_wait(&ctl.sd, ph ^ 1, ab);
                if (SAVE && c > 0) ok = ok && mbar_wait(&ctl.spfree, ph ^ 1, ab);
                if (!__all_sync(~0u, ok)) break;
                tc_fence_after();
                const float gc = gam[TC - 1];
#pragma unroll
                for (int k = 0; k < DK / 2; k += 32) {
                    float v[32];
                    tmem_ld<32>(tm + L::cS + lofs + k0 + k, v);
                    tmem_st_parts(tm + L::cP + lofs + (k0 + k) / 2, tm + L::cP + DK / 2 + lofs + (k0 + k) / 2, v);
                    uint32_t w[2][16];
#pragma unroll
                    for (int i = 0; i < 32; ++i) w[i / 16][i % 16] = __float_as_uint(gc * v[i]);
                    tmem_st16(tm + L::cS + lofs + k0 + k, w[0]);
                    tmem_st16(tm + L::cS + lofs + k0 + k + 16, w[1]);
                    tmem_st_wait();
                    tc_arrive(k == 0 ? &ctl.spa : &ctl.sp, lane);
                }
                // R = V - gamma X, tokens 32 hf ..
                const int t0 = hf * 32;
                float v[32], x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(st + L::oV + (row >> 6) * TC * 128 + (t0 + i) * 128 +
                                                                                       ((((row & 63) >> 3) ^ (i & 7)) << 4) + (row & 7) * 2)
                                           << 16);
                if (!__all_sync(~0u, mbar_wait(&ctl.xd, ph, ab))) { ok = false; break; }
                tc_fence_after();
                tmem_ld<32>(tm + L::cX + lofs + t0, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 g = *reinterpret_cast<const float4*>(gam + t0 + i);
                    v[i] = fmaf(-g.x, x[i], v[i]);
                    v[i + 1] = fmaf(-g.y, x[i + 1], v[i + 1]);
                    v[i + 2] = fmaf(-g.z, x[i + 2], v[i + 2]);
                    v[i + 3] = fmaf(-g.w, x[i + 3], v[i + 3]);
                }
                tmem_st_parts(tm + L::cR + lofs + hf * 16, tm + L::cR + 32 + lofs + hf * 16, v);
                tmem_st_wait();
                tc_arrive(&ctl.rp, lane);
                // U = beta E, and suffix U
                if (!__all_sync(~0u, mbar_wait(&ctl.ed, ph, ab))) { ok = false; break; }
                tc_fence_after();
                tmem_ld<32>(tm + L::cX + lofs + t0, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 be = *reinterpret_cast<const float4*>(gam + 2 * TC + t0 + i), su = *reinterpret_cast<const float4*>(gam + TC + t0 + i);
                    x[i] *= be.x; x[i + 1] *= be.y; x[i + 2] *= be.z; x[i + 3] *= be.w;
                    v[i] = su.x * x[i]; v[i + 1] = su.y * x[i + 1]; v[i + 2] = su.z * x[i + 2]; v[i + 3] = su.w * x[i + 3];
                }
                tmem_st_parts(tm + L::cU + lofs + hf * 16, tm + L::cU + 32 + lofs + hf * 16, v);
                tmem_st_wait();
                tc_arrive(&ctl.up, lane);
                if (!SAVE) {
                    tmem_st_parts(tm + L::cR + lofs + hf * 16, tm + L::cR + 32 + lofs + hf * 16, x);
                    tmem_st_wait();
                    tc_arrive(&ctl.ur, lane);
                }
                if (lane == 0) mbar_arrive(&ctl.empty[c % L::kStages]);
            }
            if (p.W1 && ok) {
                if (nch > 0) ok = mbar_wait(&ctl.sd, (nch - 1) & 1, ab);
                tc_fence_after();
                float* o = p.W1 + bh * state + (long long)row * DK + k0;
#pragma unroll
                for (int k = 0; k < DK / 2; k += 32) {
                    float v[32];
                    tmem_ld<32>(tm + L::cS + lofs + k0 + k, v);
                    if (ok)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(o + k + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
        } else {
            // ------------------------------------------------------------ readout (or what the backward pass keeps)
            OutRing<L::kSlots> ring{sb + L::kStages * L::stage, lane, warp == 8 && lane == 0, 0};
            for (int c = 0; c < nch; ++c) {
                const uint32_t ph = c & 1;
                const int left = len - c * TC;
                const float* gam = reinterpret_cast<const float*>(smem + (c % L::kStages) * L::stage);
                ok = full_wait(c) && mbar_wait(SAVE ? &ctl.xd : &ctl.z1, ph, ab);
                if (named_bar_or(3, 128, !ok)) break;
                tc_fence_after();
                float v[2][32];
                if (SAVE) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < DK / 64; ++k) {            // 32 columns of packed pairs: 64 values of the row
                            tmem_ld<32>(tm + L::cP + part * (DK / 2) + lofs + k * 32, v[0]);
                            if (part == 1 && k == DK / 64 - 1) tc_arrive(&ctl.spfree, lane);
                            const uint32_t slot = ring.open();
                            ring.put_row(slot, row, v[0]);
                            ring.ready();
                            if (ring.issuer) {
                                ring.store(&p.mS, slot, k * 64, (int)((((long long)bh * d.ng + c) * 2 + part) * d.dv), 0, 0);
                                bulk_commit();
                            }
                        }
                    ok = mbar_wait(&ctl.ed, ph, ab);
                    if (named_bar_or(3, 128, !ok)) break;
                    tc_fence_after();
                    tmem_ld<32>(tm + L::cX + lofs, v[0]);
                    tmem_ld<32>(tm + L::cX + lofs + 32, v[1]);
                    tc_arrive(&ctl.z2free, lane);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint32_t slot = ring.open();
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            ring.put_column(slot, row, e * 32, v[e]);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[e][i] -= lo_f(pack2(v[e][i], 0.f));
                        }
                        ring.ready();
                        if (ring.issuer) {
#pragma unroll
                            for (int k = 0; k < MV / 64; ++k) ring.store(&p.mE, slot + k * TC * 128, k * 64, c * TC, bh, part);
                            bulk_commit();
                        }
                    }
                } else {
                    tmem_ld<32>(tm + L::cZ + lofs, v[0]);
                    tmem_ld<32>(tm + L::cZ + lofs + 32, v[1]);
                    tc_arrive(&ctl.z1free, lane);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 g = *reinterpret_cast<const float4*>(gam + e * 32 + i);
                            v[e][i] *= d.scale * g.x; v[e][i + 1] *= d.scale * g.y; v[e][i + 2] *= d.scale * g.z; v[e][i + 3] *= d.scale * g.w;
                        }
                    ok = mbar_wait(&ctl.z2, ph, ab);
                    if (named_bar_or(3, 128, !ok)) break;
                    tc_fence_after();
                    float x[2][32];
                    tmem_ld<32>(tm + L::cX + lofs, x[0]);
                    tmem_ld<32>(tm + L::cX + lofs + 32, x[1]);
                    tc_arrive(&ctl.z2free, lane);
                    const uint32_t slot = ring.open();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[e][i] += v[e][i];
                        ring.put_column(slot, row, e * 32, x[e]);
                    }
                    ring.ready();
                    ring.tokens_out(&p.mZ, slot, reinterpret_cast<__nv_bfloat16*>(p.Z.p) + b * p.Z.bs + h * p.Z.hs + (long long)c * TC * p.Z.ts, p.Z.ts,
                                    c * TC, h * p.zh, b * p.zb, left, tid - 256);
                }
                if (lane == 0) mbar_arrive(&ctl.empty[c % L::kStages]);
            }
            if (ring.issuer) bulk_wait<0>();
        }
    }
    __syncthreads();
    if (warp == 13) tmem_dealloc(ctl.tmem, 512);
}

// --------------------------------------------------------------------------------------------------
// Reverse
// --------------------------------------------------------------------------------------------------
// Steps k = 0, 1, .. are the chunks from the last one.  Per step, with D the adjoint of the state:
//   D -> parts | X = D K^T, AO = dZ^T A | dU = suffix X + AO -> parts | Y = T_u^T dU | -gamma beta Y -> parts
//   D = gamma_C D + (scale gamma dZ)^T Q - (gamma beta Y)^T K
// The four output warps turn dZ into the scaled left operand one step ahead, and write D, Y and dV.
template <int DK>
struct TcReverse {
    static constexpr int oA = kTcGates, oU = oA + kTcMat, oK = oU + kTcMat, oQ = oK + DK * 128, oO = oQ + DK * 128;
    static constexpr int stage = oO + MV * 128, kStages = 2, kSlots = 3;
    static constexpr int used = kStages * stage + kSlots * MV * 128 + 512 + 1024, smem = used > 116 * 1024 ? used : 116 * 1024;   // one CTA per SM
    static_assert(smem <= 227 * 1024 && stage % 1024 == 0, "shared memory of a reverse CTA");
    static constexpr uint32_t cS = 0, cP = DK, cX = 2 * DK, cA = cX + 64, cR = cA + 64, cF = cR + 64;
};

template <int DK>
__device__ __forceinline__ void reverse_tc_body(const TcArgs& p, int bh) {
    using L = TcReverse<DK>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (s32(smem_raw) & 1023));
    const uint32_t sb = s32(smem);
    TcCtl& ctl = *reinterpret_cast<TcCtl*>(smem + L::kStages * L::stage + L::kSlots * MV * 128);
    const Dims& d = p.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = bh / d.h, h = bh % d.h;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int len = seq_len(d, b), nch = (len + TC - 1) / TC;
    const long long state = (long long)d.dv * DK;
    const Abort ab{&ctl.abort_flag, p.err, p.wait_ns};
    if (tid == 0) {
        ctl.abort_flag = 0;
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 13);
        }
        for (uint64_t* x : {&ctl.xd, &ctl.ed, &ctl.sd, &ctl.z1}) mbar_init(x, 1);
        for (uint64_t* x : {&ctl.spa, &ctl.sp, &ctl.rp, &ctl.up}) mbar_init(x, 8);
        for (uint64_t* x : {&ctl.z2free, &ctl.spfree, &ctl.fr}) mbar_init(x, 4);
        fence_barrier_init();
    }
    if (warp == 13) {
        tmem_alloc(&ctl.tmem, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tm = 0;                     // all 512 columns are this CTA's: they start at 0
    auto full_wait = [&](int k) { return mbar_wait(&ctl.full[k % L::kStages], (k / L::kStages) & 1, ab); };

    if (warp == 12) {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        int k = 0;
        for (; k < nch; ++k) {
            const int s = k % L::kStages, c = nch - 1 - k, left = len - c * TC;
            if (k >= L::kStages) ok = mbar_wait(&ctl.empty[s], (k / L::kStages - 1) & 1, ab);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            const uint32_t st = sb + s * L::stage;
            if (left < TC) {
                tok64_tail<DK>(st + L::oK, p.K, b, h / d.r, c * TC, left, lane);
                tok64_tail<DK>(st + L::oQ, p.Q, b, h / d.r, c * TC, left, lane);
                tok64_tail<MV>(st + L::oO, p.V, b, h, c * TC, left, lane);
            }
            fence_proxy_async_smem();              // the first step's stage is written by the warp, later ones by copies
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_expect_tx(&ctl.full[s], kTcGates + 2 * kTcMat + tok64_bytes<DK>(left) * 2 + tok64_bytes<MV>(left));
                const uint8_t* r = p.rec + ((long long)bh * d.nc + c) * p.rec_bytes;
                bulk_at(st, r, kTcGates, &ctl.full[s]);
                bulk_at(st + L::oA, r + kTcGates + kTcMat, 2 * kTcMat, &ctl.full[s]);
                if (left >= TC) {
                    tok64_load<DK>(st + L::oK, p.K, &ctl.full[s], b, h / d.r, c * TC);
                    tok64_load<MV>(st + L::oO, p.V, &ctl.full[s], b, h, c * TC);
                    tok64_load<DK>(st + L::oQ, p.Q, &ctl.full[s], b, h / d.r, c * TC);
                }
            }
            __syncwarp();
        }
        for (int i = max(0, k - L::kStages); i < k; ++i) mbar_drain(&ctl.full[i % L::kStages], (i / L::kStages) & 1, drain_limit(ab));
    } else if (warp == 13) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t id64 = idesc_bf16_f32(MV, 64, false, false), idS = idesc_bf16_f32(MV, DK, false, true);
        bool ok = true;
        int k = 0;
        for (; k < nch; ++k) {
            const uint32_t ph = k & 1, st = sb + (k % L::kStages) * L::stage;
            ok = __all_sync(~0u, full_wait(k));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {                     // tokens i of 16 kk .. reach columns j up to 16 kk + 15 of A
#pragma unroll
                for (int kk = 3; kk >= 0; --kk) {
                    const uint32_t id = idesc_bf16_f32(MV, 16, true, true) + ((uint32_t)kk * 2 << 17);     // N = 16 (kk + 1)
                    const uint64_t a = sdesc_sw128(st + L::oO + kk * 2048, TC * 128, 1024);
                    mma_bf16_ss(tm + L::cA, a, sdesc_sw128(st + L::oA + kk * 2048, TC * 128, 1024), id, kk < 3);
                    mma_bf16_ss(tm + L::cA, a, sdesc_sw128(st + L::oA + TC * 128 + kk * 2048, TC * 128, 1024), id, 1);
                }
            }
            __syncwarp();
            ok = mbar_wait(&ctl.spa, ph, ab);
            if (k > 0) ok = ok && mbar_wait(&ctl.z2free, ph ^ 1, ab);          // Y has been read out
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            state_product<DK>(tm + L::cX, tm + L::cP, st + L::oK, id64, 0);
            if (DK == 128) {
                ok = __all_sync(~0u, mbar_wait(&ctl.sp, ph, ab));
                if (!ok) break;
                tc_fence_after();
                state_product<DK>(tm + L::cX, tm + L::cP, st + L::oK, id64, 1);
            }
            if (elect_one()) mma_commit(&ctl.xd);
            __syncwarp();
            ok = __all_sync(~0u, mbar_wait(&ctl.rp, ph, ab));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 3; kk >= 0; --kk) {
                    const uint32_t id = idesc_bf16_f32(MV, 16, false, true) + ((uint32_t)kk * 2 << 17);
                    const uint64_t hi = sdesc_sw128(st + L::oU + kk * 2048, TC * 128, 1024), lo = sdesc_sw128(st + L::oU + TC * 128 + kk * 2048, TC * 128, 1024);
                    mma_bf16_ts(tm + L::cX, tm + L::cR + kk * 8, hi, id, kk < 3);
                    mma_bf16_ts(tm + L::cX, tm + L::cR + kk * 8, lo, id, 1);
                    mma_bf16_ts(tm + L::cX, tm + L::cR + 32 + kk * 8, hi, id, 1);
                }
                mma_commit(&ctl.ed);
            }
            __syncwarp();
            auto outer = [&](uint32_t a, uint32_t x) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        mma_bf16_ts(tm + L::cS, a + part * 32 + kk * 8, sdesc_sw128(x + kk * 2048, TC * 128, 1024), idS, 1);
            };
            ok = __all_sync(~0u, mbar_wait(&ctl.fr, ph, ab));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                outer(tm + L::cF, st + L::oQ);
                mma_commit(&ctl.z1);
            }
            __syncwarp();
            ok = __all_sync(~0u, mbar_wait(&ctl.up, ph, ab));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                outer(tm + L::cR, st + L::oK);
                mma_commit(&ctl.sd);
                mma_commit(&ctl.empty[k % L::kStages]);
            }
            __syncwarp();
        }
        // the last products end before the CTA gives its tensor memory back
        if (!ok) {
            if (elect_one()) mma_commit(&ctl.sd);
            __syncwarp();
            mbar_drain(&ctl.sd, k & 1, drain_limit(ab));
        } else if (nch > 0) {
            mbar_drain(&ctl.sd, (nch - 1) & 1, drain_limit(ab));
        }
    } else {
        const int q = warp & 3;
        const uint32_t lofs = (uint32_t)(q * 32) << 16;
        const int row = q * 32 + lane;
        bool ok = true;
        if (warp < 8) {
            // ------------------------------------------------------------ chain
            const int hf = warp >> 2, k0 = hf * (DK / 2);
            const float* w0 = p.W0 ? p.W0 + b * p.w0_bs + h * state + (long long)row * DK + k0 : nullptr;
#pragma unroll
            for (int j = 0; j < DK / 2; j += 16) {
                uint32_t r[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 v = w0 ? *reinterpret_cast<const float4*>(w0 + j + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    r[i] = __float_as_uint(v.x); r[i + 1] = __float_as_uint(v.y); r[i + 2] = __float_as_uint(v.z); r[i + 3] = __float_as_uint(v.w);
                }
                tmem_st16(tm + L::cS + lofs + k0 + j, r);
            }
            tmem_st_wait();
            for (int k = 0; k < nch; ++k) {
                const uint32_t ph = k & 1;
                const float* gam = reinterpret_cast<const float*>(smem + (k % L::kStages) * L::stage);
                ok = full_wait(k);
                if (k > 0) ok = ok && mbar_wait(&ctl.sd, ph ^ 1, ab) && mbar_wait(&ctl.spfree, ph ^ 1, ab);
                if (!__all_sync(~0u, ok)) break;
                tc_fence_after();
                const float gc = gam[TC - 1];
#pragma unroll
                for (int j = 0; j < DK / 2; j += 32) {
                    float v[32];
                    tmem_ld<32>(tm + L::cS + lofs + k0 + j, v);
                    tmem_st_parts(tm + L::cP + lofs + (k0 + j) / 2, tm + L::cP + DK / 2 + lofs + (k0 + j) / 2, v);
                    uint32_t w[2][16];
#pragma unroll
                    for (int i = 0; i < 32; ++i) w[i / 16][i % 16] = __float_as_uint(gc * v[i]);
                    tmem_st16(tm + L::cS + lofs + k0 + j, w[0]);
                    tmem_st16(tm + L::cS + lofs + k0 + j + 16, w[1]);
                    tmem_st_wait();
                    tc_arrive(j == 0 ? &ctl.spa : &ctl.sp, lane);
                }
                const int t0 = hf * 32;
                float v[32], x[32];
                if (!__all_sync(~0u, mbar_wait(&ctl.xd, ph, ab))) { ok = false; break; }
                tc_fence_after();
                tmem_ld<32>(tm + L::cX + lofs + t0, x);
                tmem_ld<32>(tm + L::cA + lofs + t0, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 s = *reinterpret_cast<const float4*>(gam + TC + t0 + i);
                    v[i] = fmaf(s.x, x[i], v[i]);
                    v[i + 1] = fmaf(s.y, x[i + 1], v[i + 1]);
                    v[i + 2] = fmaf(s.z, x[i + 2], v[i + 2]);
                    v[i + 3] = fmaf(s.w, x[i + 3], v[i + 3]);
                }
                tmem_st_parts(tm + L::cR + lofs + hf * 16, tm + L::cR + 32 + lofs + hf * 16, v);
                tmem_st_wait();
                tc_arrive(&ctl.rp, lane);
                if (!__all_sync(~0u, mbar_wait(&ctl.ed, ph, ab))) { ok = false; break; }
                tc_fence_after();
                tmem_ld<32>(tm + L::cX + lofs + t0, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 g = *reinterpret_cast<const float4*>(gam + t0 + i), be = *reinterpret_cast<const float4*>(gam + 2 * TC + t0 + i);
                    x[i] *= -g.x * be.x; x[i + 1] *= -g.y * be.y; x[i + 2] *= -g.z * be.z; x[i + 3] *= -g.w * be.w;
                }
                tmem_st_parts(tm + L::cR + lofs + hf * 16, tm + L::cR + 32 + lofs + hf * 16, x);
                tmem_st_wait();
                tc_arrive(&ctl.up, lane);
                if (lane == 0) mbar_arrive(&ctl.empty[k % L::kStages]);
            }
            if (p.W1 && ok) {
                if (nch > 0) ok = mbar_wait(&ctl.sd, (nch - 1) & 1, ab);
                tc_fence_after();
                float* o = p.W1 + bh * state + (long long)row * DK + k0;
#pragma unroll
                for (int j = 0; j < DK / 2; j += 32) {
                    float v[32];
                    tmem_ld<32>(tm + L::cS + lofs + k0 + j, v);
                    if (ok)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(o + j + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
        } else {
            // ------------------------------------------------------------ scaled dZ, and what the step gives
            OutRing<L::kSlots> ring{sb + L::kStages * L::stage, lane, warp == 8 && lane == 0, 0};
            // scale gamma dZ of step k, as parts
            auto scaled = [&](int k) {
                const int left = len - (nch - 1 - k) * TC;
                const uint8_t* st = smem + (k % L::kStages) * L::stage;
                const float* gam = reinterpret_cast<const float*>(st);
                ok = full_wait(k);
                if (k > 0) ok = ok && mbar_wait(&ctl.z1, (k - 1) & 1, ab);     // the step before has used its own
                if (named_bar_or(3, 128, !ok)) return false;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const uint32_t x = *reinterpret_cast<const uint16_t*>(st + L::oO + (row >> 6) * TC * 128 + (e * 32 + i) * 128 +
                                                                               ((((row & 63) >> 3) ^ (i & 7)) << 4) + (row & 7) * 2);
                        v[i] = e * 32 + i < left ? __uint_as_float(x << 16) * (d.scale * gam[e * 32 + i]) : 0.f;
                    }
                    tmem_st_parts(tm + L::cF + lofs + e * 16, tm + L::cF + 32 + lofs + e * 16, v);
                }
                tmem_st_wait();
                tc_arrive(&ctl.fr, lane);
                return true;
            };
            bool go = nch > 0 && scaled(0);
            for (int k = 0; go && k < nch; ++k) {
                const uint32_t ph = k & 1;
                const int c = nch - 1 - k, left = len - c * TC;
                const float* gam = reinterpret_cast<const float*>(smem + (k % L::kStages) * L::stage);
                float v[2][32];
                ok = mbar_wait(&ctl.xd, ph, ab);
                if (named_bar_or(3, 128, !ok)) break;
                tc_fence_after();
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int j = 0; j < DK / 64; ++j) {
                        tmem_ld<32>(tm + L::cP + part * (DK / 2) + lofs + j * 32, v[0]);
                        if (part == 1 && j == DK / 64 - 1) tc_arrive(&ctl.spfree, lane);
                        const uint32_t slot = ring.open();
                        ring.put_row(slot, row, v[0]);
                        ring.ready();
                        if (ring.issuer) {
                            ring.store(&p.mS, slot, j * 64, (int)((((long long)bh * d.ng + c) * 2 + part) * d.dv), 0, 0);
                            bulk_commit();
                        }
                    }
                if (k + 1 < nch && !(go = scaled(k + 1))) break;
                ok = mbar_wait(&ctl.ed, ph, ab);
                if (named_bar_or(3, 128, !ok)) break;
                tc_fence_after();
                tmem_ld<32>(tm + L::cX + lofs, v[0]);
                tmem_ld<32>(tm + L::cX + lofs + 32, v[1]);
                tc_arrive(&ctl.z2free, lane);
                {
                    const uint32_t slot = ring.open();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = gam[2 * TC + e * 32 + i] * v[e][i];
                        ring.put_column(slot, row, e * 32, x);
                    }
                    ring.ready();
                    ring.tokens_out(&p.mZ, slot, reinterpret_cast<__nv_bfloat16*>(p.Z.p) + b * p.Z.bs + h * p.Z.hs + (long long)c * TC * p.Z.ts, p.Z.ts,
                                    c * TC, h * p.zh, b * p.zb, left, tid - 256);
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint32_t slot = ring.open();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ring.put_column(slot, row, e * 32, v[e]);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[e][i] -= lo_f(pack2(v[e][i], 0.f));
                    }
                    ring.ready();
                    if (ring.issuer) {
#pragma unroll
                        for (int j = 0; j < MV / 64; ++j) ring.store(&p.mE, slot + j * TC * 128, j * 64, c * TC, bh, part);
                        bulk_commit();
                    }
                }
                if (lane == 0) mbar_arrive(&ctl.empty[k % L::kStages]);
            }
            if (ring.issuer) bulk_wait<0>();
        }
    }
    __syncthreads();
    if (warp == 13) tmem_dealloc(ctl.tmem, 512);
}

template <int DK>
__global__ void __launch_bounds__(448, 1) delta_chain_tc(const __grid_constant__ TcArgs p) {
    chain_tc_body<DK, false>(p, blockIdx.x);
}
// The backward pass's two sequential sweeps need nothing of each other: one launch, the longer ones first.
template <int DK>
__global__ void __launch_bounds__(448, 1) delta_both_tc(const __grid_constant__ TcArgs chain, const __grid_constant__ TcArgs reverse) {
    const int n = chain.d.B * chain.d.h;
    if ((int)blockIdx.x < n) reverse_tc_body<DK>(reverse, blockIdx.x);
    else chain_tc_body<DK, true>(chain, blockIdx.x - n);
}

// --------------------------------------------------------------------------------------------------
// Launches
// --------------------------------------------------------------------------------------------------
static bool map64(Tok64* t, const Parts& x, const Dims& d, int heads, int width) {
    t->p = x.p;
    t->bs = x.bs; t->hs = x.hs; t->ts = x.ts;
    t->hmul = x.hs != 0;
    t->bmul = x.bs != 0;
    return (x.ts != 0 || d.N == 1) &&
           encode_map(&t->map, x.p, 2, {(cuuint64_t)width, (cuuint64_t)d.N, (cuuint64_t)(x.hs ? heads : 1), (cuuint64_t)(x.bs ? d.B : 1), 1},
                      {x.ts ? x.ts : width, x.hs ? x.hs : width, x.bs ? x.bs : width, width}, 128, TC);
}
static Parts bf16_parts(const View& x) { return Parts{reinterpret_cast<const __nv_bfloat16*>(x.p), 0, x.bs, x.hs, x.ts}; }

// The arguments every tensor-core kernel of a call shares; false where a token tensor has no tensor map (a token
// stride of zero).
static bool tc_args(TcArgs* a, const Call& c, bool backward, uint8_t* rec) {
    a->d = c.d;
    a->d.nc = (c.d.N + TC - 1) / TC;
    a->rec = rec;
    a->rec_bytes = tc_rec_bytes(backward);
    a->err = error_word(c);
    a->wait_ns = c.wait_ns;
    return map64(&a->K, bf16_parts(c.K), c.d, c.d.hk, c.d.dk) && map64(&a->Q, bf16_parts(c.Q), c.d, c.d.hk, c.d.dk) &&
           map64(&a->V, bf16_parts(c.V), c.d, c.d.h, c.d.dv);
}
// The maps of a kernel's outputs: Z (or dV), and in the backward pass E (or Y) and the states (or adjoints).
static bool tc_outputs(TcArgs* a, const View& z, const Dims& d, __nv_bfloat16* E, long long e_ps, __nv_bfloat16* S) {
    a->Z = z;
    a->zh = z.hs != 0;
    a->zb = z.bs != 0;
    bool ok = encode_map(&a->mZ, z.p, 2, {(cuuint64_t)d.dv, (cuuint64_t)d.N, (cuuint64_t)(z.hs ? d.h : 1), (cuuint64_t)(z.bs ? d.B : 1), 1},
                         {z.ts ? z.ts : d.dv, z.hs ? z.hs : d.dv, z.bs ? z.bs : d.dv, d.dv}, 128, TC);
    if (E) {
        const long long srows = (long long)d.B * d.h * d.ng * 2 * d.dv;
        ok = ok && srows < (1LL << 31) &&
             encode_map(&a->mE, E, 2, {(cuuint64_t)d.dv, (cuuint64_t)d.N, (cuuint64_t)d.B * d.h, 2, 1}, {d.dv, (long long)d.N * d.dv, e_ps, e_ps}, 128, TC) &&
             encode_map2(&a->mS, S, d.dk, srows, d.dv);
    }
    return ok;
}
template <int DK, bool BACKWARD>
static ttt_status run_prep64(const Call& c, uint8_t* rec) {
    using L = Prep64<DK, BACKWARD>;
    constexpr auto k = delta_prep64<DK, BACKWARD>;
    ttt_status st = allow_smem<k>(L::smem);
    if (st != TTT_OK) return st;
    const long long n = (long long)c.d.B * c.d.h * ((c.d.N + TC - 1) / TC);
    return launch(k, n, 128, L::smem, c.stream, c.d, bf16_parts(c.Q), bf16_parts(c.K), c.G, c.Beta, rec, error_word(c));
}
template <int DK>
static ttt_status run_chain_tc(const Call& c, const TcArgs& a) {
    constexpr auto k = delta_chain_tc<DK>;
    constexpr int smem = TcChain<DK, false>::smem;
    const ttt_status st = allow_smem<k>(smem);
    return st != TTT_OK ? st : launch(k, c.d.B * c.d.h, 448, smem, c.stream, a);
}
template <int DK>
static ttt_status run_both_tc(const Call& c, const TcArgs& chain, const TcArgs& reverse) {
    constexpr auto k = delta_both_tc<DK>;
    constexpr int smem = std::max(TcChain<DK, true>::smem, TcReverse<DK>::smem);
    const ttt_status st = allow_smem<k>(smem);
    return st != TTT_OK ? st : launch(k, 2LL * c.d.B * c.d.h, 448, smem, c.stream, chain, reverse);
}
