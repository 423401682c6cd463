// delta.cu -- the gated delta rule over whole sequences: forward pass and the states it passes through.
//
//   W_t = e^{g_t} W_{t-1} + beta_t (v_t - e^{g_t} W_{t-1} k_t) k_t^T,   z_t = scale W_t q_t
//
// Chunks of C = 32 tokens.  With gamma_i = exp(g_1 + .. + g_i) inside a chunk, Gamma_ij = exp(g_{j+1} + .. +
// g_i) for j <= i and G_ij = Gamma_ij k_i.k_j for j < i, the residuals e_i = v_i - e^{g_i} W_{i-1} k_i of a
// chunk that starts from W solve (I + G diag(beta)) E = V - diag(gamma) K W^T.  So
//   prep   (one warp per image, value head and chunk, all at once):
//          T' = (I + G diag(beta))^{-1}, A = scale Gamma .* (Q K^T) for j <= i;
//   chain  (a warp per 16 rows of W, sequential over the chunks):
//          R = V - diag(gamma) K W^T,  E = T' R,  U = diag(beta) E,
//          Z = scale diag(gamma) Q W^T + A U,   W <- gamma_C W + U^T diag(Gamma_C.) K.
// Every sum of log gates starts at zero (no difference of two long prefix sums), so a gate of -inf
// (a state that is dropped) and strong gates keep their accuracy.
//
// The chain's rows are independent, so that a warp that owns 16 rows of W keeps them in registers as
// the accumulators of U^T K, and each product's accumulators are the next one's left operand (the
// m16n8k16 accumulator and A-operand layouts agree after a pack to bf16): W -> K W^T -> E -> W never waits on another
// warp within a chunk, but for one: two warps share 16 rows, each with half of d_k, and add up their halves of K W^T through
// shared memory (KS = 2).  A loader warp brings the token tiles by TMA a chunk or two ahead, and helper warps
// take the readout and the stores, one chunk behind.  One warp for 16 rows against two: forward, 32 heads of 8192 tokens, d = 128,
// 638 us against 488, 48 heads of 6084, d = 64, 337 against 297; backward, 32 heads of 4096, d = 128, 1224 against 1070.
//
// Precision: W and all sums are fp32.  An operand of a matrix instruction that no bf16 value holds (W, R, E, U, T', A; fp32 tokens, by a
// pass of their own) is split into three bf16 parts, 24 bits, products of parts below the third dropped.  The matrix instructions
// truncate: each of an instruction's products is cut at a quarter of the last place of the largest addend, and the sum towards zero.
// So sums of many products are taken in accumulators of their own, the small products first or apart, and added to the rest in fp32.
// 2-norm errors, d = 64 .. 128, gates of 0 .. -3: W1 1 to 2e-7, fp32 Z 2e-7, gradients in fp32 1 to 5e-7; a plain fp32 computation in
// chunks: 1 to 4e-7.  (Two parts for R or suffix U alone: W1 2.4e-6, 2.6e-6; two in the readout, 5 to 10 % faster: Z 3e-6 before its rounding.)
//
// Bound: the chain of chunks, about 3,300 cycles for 32 tokens at d = 128 (matrix instructions, measured at 1,009
// multiply-adds per cycle and SM, about half of it; the rest is their latency and shared-memory reads of the token
// operands).  32 heads of 8192 tokens, d = 128, two value heads to a key head: prep 55 us, chain 435 us.
#include <algorithm>
#include <array>
#include <atomic>

#include "delta.cuh"

namespace ttt {
namespace gd {

// --------------------------------------------------------------------------------------------------
// fp32 tokens -> bf16 parts, contiguous [part][B][heads][N][width]
// --------------------------------------------------------------------------------------------------
struct SplitArgs {
    View x[3];
    __nv_bfloat16* out[3];
    long long ps[3];                  // elements of a tensor = part stride
    int heads[3], width[3];
    Dims d;
};
__global__ void __launch_bounds__(256) split_tokens(const __grid_constant__ SplitArgs a) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const int i = blockIdx.y, w4 = a.width[i] / 4, heads = a.heads[i];
    const long long total = a.ps[i] / 4;
    for (long long x = blockIdx.x * 256LL + threadIdx.x; x < total; x += gridDim.x * 256LL) {
        const int c = (int)(x % w4) * 4;
        const long long row = x / w4;
        const int bh = (int)(row / a.d.N), t = (int)(row - (long long)bh * a.d.N), b = bh / heads, h = bh - b * heads;
        if (t >= seq_len(a.d, b)) continue;            // what lies behind a sequence is not read
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.x[i].p) + b * a.x[i].bs + h * a.x[i].hs +
                                                          t * a.x[i].ts + c);
        uint32_t lo[P], hi[P];
        split2(v.x, v.y, lo);
        split2(v.z, v.w, hi);
#pragma unroll
        for (int p = 0; p < P; ++p) *reinterpret_cast<uint2*>(a.out[i] + p * a.ps[i] + row * a.width[i] + c) = make_uint2(lo[p], hi[p]);
    }
}

// --------------------------------------------------------------------------------------------------
// Prep
// --------------------------------------------------------------------------------------------------
constexpr int GP = CT + 4;            // row pitch (floats) of the 32 x 32 fp32 matrices of a warp

// Warps (chunks) per CTA.  Bound: issue and latency of about 2,000 instructions per warp with 3 TB/s of reads and records beside them.
// Shared memory (59 KB a CTA) keeps three CTAs, twelve warps, on an SM.
constexpr int kPrepWarps = 4;
// A warp's shared memory: Gamma, then G in its place, one matrix image, and two 16 x 16 blocks.
constexpr int kPrepWarpBytes = CT * GP * 4 + kMat + 2 * 16 * 20 * 4;

// The lower triangles of K K^T (c) and Q K^T (w) of 32 tokens, rows behind `left` as zeros.  The operands go from global
// memory to registers: any order of the features does as long as both sides have it, so that a lane takes 8
// in a row, which are its operands of two products (each row of K being a left and a right operand).
template <int DK, int PK>
__device__ __forceinline__ void gram32(float (&c)[2][4][4], float (&w)[2][4][4], const Parts& K, const Parts& Q, long long ko, long long qo,
                                       int left, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) c[m][n][q] = w[m][n][q] = 0.f;
#pragma unroll(PK == 1 ? 2 : 1)
    for (int f = 0; f < DK; f += 32) {
        uint4 k[PK][4], q[PK][4];
#pragma unroll
        for (int p = 0; p < PK; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = g + 8 * i;
                const bool live = row < left;
                k[p][i] = live ? *reinterpret_cast<const uint4*>(K.p + p * K.ps + ko + row * K.ts + f + t * 8) : make_uint4(0, 0, 0, 0);
                q[p][i] = live ? *reinterpret_cast<const uint4*>(Q.p + p * Q.ps + qo + row * Q.ts + f + t * 8) : make_uint4(0, 0, 0, 0);
            }
        // more than one part: the products of a block are summed in accumulators of their own, the small ones first
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 2 * m + 2; ++n) {
                float uc[4] = {}, uw[4] = {};
#pragma unroll
                for (int order = PK - 1; order >= 0; --order)
#pragma unroll
                    for (int pb = 0; pb < PK; ++pb) {
                        const int pa = order - pb;
                        if (pa < 0) continue;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            auto lo = [&](const uint4& v) { return half ? v.z : v.x; };
                            auto hi = [&](const uint4& v) { return half ? v.w : v.y; };
                            const uint32_t ak[4] = {lo(k[pa][2 * m]), lo(k[pa][2 * m + 1]), hi(k[pa][2 * m]), hi(k[pa][2 * m + 1])};
                            const uint32_t aq[4] = {lo(q[pa][2 * m]), lo(q[pa][2 * m + 1]), hi(q[pa][2 * m]), hi(q[pa][2 * m + 1])};
                            mma16816(PK > 1 ? uc : c[m][n], ak, lo(k[pb][n]), hi(k[pb][n]));
                            mma16816(PK > 1 ? uw : w[m][n], aq, lo(k[pb][n]), hi(k[pb][n]));
                        }
                    }
                if (PK > 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        c[m][n][e] += uc[e];
                        w[m][n][e] += uw[e];
                    }
            }
    }
}

// Elements (i, j) and (i, j + 1), j even, of a bf16 part image.
__device__ __forceinline__ void put_parts2(uint8_t* mat, int i, int j, float x, float y) {
    uint32_t w[P];
    split2(x, y, w);
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<uint32_t*>(mat + ((p * CT + i) * MP + j) * 2) = w[p];
}

// The warp's matrix image in shared memory -> global memory.
__device__ __forceinline__ void copy_image(uint8_t* dst, const uint8_t* image, int lane) {
    __syncwarp();
#pragma unroll
    for (int x = lane; x < kMat / 16; x += 32) reinterpret_cast<uint4*>(dst)[x] = reinterpret_cast<const uint4*>(image)[x];
    __syncwarp();
}
constexpr int XP = 20, kBlock = 16 * XP;   // row pitch and size (floats) of a 16 x 16 block

// The image of (I + G diag(beta))^{-1} (U: of (I + diag(beta) G)^{-1}), G 32 x 32, strictly lower triangular.  The two 16 x 16
// blocks on the diagonal are inverted by forward substitution, a column per lane; the block below them is
// - T_22 L_21 T_11 on matrix instructions, whose operands are P parts as the image's elements are.
template <bool U>
__device__ __forceinline__ void inverse_image(uint8_t* image, const float* gm, float* blocks, float beta, int lane) {
    {
        const int half = lane >> 4, col = lane & 15;
        const float* gh = gm + half * 16 * (GP + 1);
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int l = 0; l < 16; l += 4) {
                if (l >= i) continue;
                const float4 v = *reinterpret_cast<const float4*>(gh + i * GP + l);
                s[0] = fmaf(v.x, y[l], s[0]);
                if (l + 1 < i) s[1] = fmaf(v.y, y[l + 1], s[1]);
                if (l + 2 < i) s[2] = fmaf(v.z, y[l + 2], s[2]);
                if (l + 3 < i) s[3] = fmaf(v.w, y[l + 3], s[3]);
            }
            const float be = __shfl_sync(~0u, beta, half * 16 + i), sum = (s[0] + s[1]) + (s[2] + s[3]);
            const float x = i < col ? 0.f : (i == col ? 1.f : 0.f) - (U ? be * sum : sum);
            blocks[half * kBlock + i * XP + col] = x;
            y[i] = U ? x : be * x;
        }
    }
    __syncwarp();
    const int g = lane >> 2, t = lane & 3;
    // A row of L_21 that is not finite (or beyond bf16's range) must not reach the rows before it through the zeros of T_22: it
    // counts as zero, and rows from the first one on are NaN.
    auto beyond = [](float v) { return !(fabsf(v) < 3.39e38f); };
    int bad = 32;
    uint32_t m[P][4];                              // T_22 L_21, its accumulators as the next left operand
    {
        uint32_t a[P][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 v = *reinterpret_cast<const float2*>(blocks + kBlock + (g + (e & 1) * 8) * XP + 2 * t + (e >> 1) * 8);
            uint32_t w[P];
            split2(v.x, v.y, w);
#pragma unroll
            for (int p = 0; p < P; ++p) a[p][e] = w[p];
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint32_t b[P][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = 16 + 2 * t + e * 8;
                const float f0 = __shfl_sync(~0u, beta, U ? k : n * 8 + g), f1 = __shfl_sync(~0u, beta, U ? k + 1 : n * 8 + g);
                float l0 = f0 * gm[k * GP + n * 8 + g], l1 = f1 * gm[(k + 1) * GP + n * 8 + g];
                if (beyond(l1)) { bad = min(bad, k + 1); l1 = 0.f; }
                if (beyond(l0)) { bad = min(bad, k); l0 = 0.f; }
                uint32_t w[P];
                split2(l0, l1, w);
#pragma unroll
                for (int p = 0; p < P; ++p) b[p][e] = w[p];
            }
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int pa = 0; pa < P; ++pa)
#pragma unroll
                for (int pb = 0; pa + pb < P; ++pb) mma16816(c, a[pa], b[pb][0], b[pb][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t w[P];
                split2(c[2 * e], c[2 * e + 1], w);
#pragma unroll
                for (int p = 0; p < P; ++p) m[p][2 * n + e] = w[p];
            }
        }
    }
    bad = __reduce_min_sync(~0u, bad);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        uint32_t b[P][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float* x = blocks + (2 * t + e * 8) * XP + n * 8 + g;
            uint32_t w[P];
            split2(x[0], x[XP], w);
#pragma unroll
            for (int p = 0; p < P; ++p) b[p][e] = w[p];
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int pa = 0; pa < P; ++pa)
#pragma unroll
            for (int pb = 0; pa + pb < P; ++pb) mma16816(c, m[pa], b[pb][0], b[pb][1]);
        const float low = 16 + g >= bad ? __int_as_float(0x7fffffff) : 0.f, high = 24 + g >= bad ? __int_as_float(0x7fffffff) : 0.f;
        put_parts2(image, 16 + g, n * 8 + 2 * t, low - c[0], low - c[1]);
        put_parts2(image, 24 + g, n * 8 + 2 * t, high - c[2], high - c[3]);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int block = r >> 2, i = (r & 3) * 4 + (lane >> 3), j = (lane & 7) * 2;
        const float2 v = *reinterpret_cast<const float2*>(blocks + block * kBlock + i * XP + j);
        put_parts2(image, block * 16 + i, block * 16 + j, v.x, v.y);
    }
}

template <int DK, int PK, bool BACKWARD>
__global__ void __launch_bounds__(kPrepWarps * 32, PK == 1 ? 3 : 2)
delta_prep(Dims d, Parts Q, Parts K, View G, View Beta, uint8_t* rec, long long total, uint32_t* err) {
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long item = (long long)blockIdx.x * kPrepWarps + warp;
    if (blockIdx.x == 0 && threadIdx.x == 0) *err = 0;
    if (item >= total) return;
    const int c = (int)(item % d.nc);
    const long long bh = item / d.nc;
    const int h = (int)(bh % d.h), b = (int)(bh / d.h);
    const int left = seq_len(d, b) - c * CT;
    if (left <= 0) return;
    uint8_t* my = smem + warp * kPrepWarpBytes;
    float* kkm = reinterpret_cast<float*>(my);
    uint8_t* image = my + CT * GP * 4;
    float* blocks = reinterpret_cast<float*>(image + kMat);
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
    uint8_t* out = rec + item * rec_bytes(BACKWARD);
    float* gates = reinterpret_cast<float*>(out);
    gates[lane] = expf(pre);
    gates[CT + lane] = expf(suf);
    gates[2 * CT + lane] = beta;

    {
        // column `lane` (= j): Gamma_ij with its log summed from zero at i = j
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const float gi = __shfl_sync(~0u, g, i);
            s = i > lane ? s + gi : 0.f;
            kkm[i * GP + lane] = i < lane ? 0.f : expf(s);
        }
    }
    __syncwarp();
    {
        float m[2][4][4], w[2][4][4];
        gram32<DK, PK>(m, w, K, Q, b * K.bs + (h / d.r) * K.hs + (long long)c * CT * K.ts, b * Q.bs + (h / d.r) * Q.hs + (long long)c * CT * Q.ts,
                       left, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = x * 16 + (lane >> 2) + e * 8, j = n * 8 + 2 * (lane & 3);
                    if (n > 2 * x + 1) {                       // above the diagonal (G is zero there already)
                        put_parts2(image, i, j, 0.f, 0.f);
                        continue;
                    }
                    const bool edge = n >= 2 * x;              // the diagonal may pass: nothing above it may come through, NaN neither
                    float2* dec = reinterpret_cast<float2*>(kkm + i * GP + j);
                    const float2 gm = *dec;
                    put_parts2(image, i, j, edge && j > i ? 0.f : d.scale * gm.x * w[x][n][2 * e],
                                  edge && j + 1 > i ? 0.f : d.scale * gm.y * w[x][n][2 * e + 1]);
                    *dec = make_float2(edge && j >= i ? 0.f : gm.x * m[x][n][2 * e], edge && j + 1 >= i ? 0.f : gm.y * m[x][n][2 * e + 1]);
                }
    }
    copy_image(out + kGateBytes + kMat, image, lane);
    inverse_image<false>(image, kkm, blocks, beta, lane);  // what lies above the diagonal is zero from A on
    copy_image(out + kGateBytes, image, lane);
    if constexpr (BACKWARD) {
        inverse_image<true>(image, kkm, blocks, beta, lane);
        copy_image(out + kGateBytes + 2 * kMat, image, lane);
    }
}

// --------------------------------------------------------------------------------------------------
// Chain
// --------------------------------------------------------------------------------------------------
// A tile is 16 state rows, and two helpers finish it.  With at most one tile per SM (over the sweeps of the launch: one forward, two in the
// backward pass) a CTA takes one tile, else two, which share the token tiles in shared memory.  2048 tokens, d = 128, forward by one / by
// two: 144 tiles 106 / 122 us, 192 tiles 197 / 123; backward, tiles of each sweep: 72 248 / 271, 80 308 / 303, 144 382 / 359, 256 690 / 556.
static bool few_tiles(const Call& c, int sweeps) { return (long long)c.d.B * c.d.h * (c.d.dv / 16) * sweeps <= c.sms; }

struct ChainOut {
    View Z;                       // forward: the readout
    float* W1;                    // nullable [B][h][dv][dk]
    __nv_bfloat16* E;             // backward: residual parts [P][B][h][N][dv]
    long long e_ps;
    __nv_bfloat16* S;             // backward: states at the groups' starts [B][h][ng][P][dv][dk]
};

// A CTA of a sequential kernel: RT tiles of 16 rows of the state.  Chain warps: KS per tile, each owning DK / KS
// of the tile's columns.  Helper warps: kHelp per tile, off the sequential path.  One warp loads.
// The CTA goes from period to period with one barrier each.
constexpr int kHelp = 2;
constexpr int kGateSlots = 8;                                  // chunks whose gates are kept in shared memory
template <int RT, int KS>
__host__ __device__ constexpr int seq_warps() { return RT * KS + RT * kHelp + 1; }

// Control block of a sequential kernel's CTA.
struct Ctl {
    uint64_t full[4];
    int abort_flag;
};
constexpr int kCtlBytes = 64;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

template <int DK, int PK, int RT, int KS, bool SAVE>
struct ChainLayout {
    static constexpr int VW = RT * 16;
    static constexpr int VB = VW * (PK == 1 ? 2 : 4);          // bytes of a row of the value tile
    static constexpr int kK = PK * CT * DK * 2;                // K of the period's chunk, then Q of the one before
    static constexpr int kQ = SAVE ? 0 : kK;
    static constexpr int kV = CT * VB;
    static constexpr int kT = kMat, kA = SAVE ? 0 : kMat;     // T', then A of the chunk before
    static constexpr int stage = (kK + kQ + kV + kT + kA + 1023) / 1024 * 1024;
    static constexpr int kGates = kGateSlots * kGateBytes;
    static constexpr int kS = DK / 16 * P * 512;               // a tile's state as operand parts
    static constexpr int kE = 2048;                            // a tile's residuals (or partial sums), fp32
    static constexpr int kX = KS > 1 ? RT * KS * kE : 0;
    static constexpr int kOut = RT * kHelp * P * 16 * 48;      // 16 tokens x 16 values per helper and part, pitch 24
    static constexpr int fixed = kCtlBytes + kGates + 2 * RT * (kS + kE) + kX + kOut + 1024;   // 1024: alignment
    static constexpr int kStages = 3 * stage + fixed <= 227 * 1024 ? 3 : 2;
    static constexpr int smem = kStages * stage + fixed;
    static_assert(VB <= 128 && kK % 1024 == 0 && kV % 1024 == 0, "swizzled tiles");
};

// acc (16 x 8) += (PA parts a of 16 rows x 32 k) * B for one block nb of 8 columns, B a lower-triangular matrix image
// [P][32][MP]; the products of the smallest parts first.  NT: B[k][n] = M[n][k] (columns n of the product are M's
// rows);  else B[k][n] = M[k][n].
template <int PA, bool NT>
__device__ __forceinline__ void mat_block(float (&acc)[4], const uint32_t (&a)[2][PA][4], uint32_t mat, int nb, int lane) {
    const int mi = lane >> 3, lr = lane & 7;
    uint32_t b[P][4];
#pragma unroll
    for (int pb = 0; pb < P; ++pb) {
        if (NT) ldsm4(b[pb], mat + ((pb * CT + nb * 8 + lr) * MP + mi * 8) * 2);
        else ldsm4t(b[pb], mat + ((pb * CT + mi * 8 + lr) * MP + nb * 8) * 2);
    }
#pragma unroll
    for (int order = P - 1; order >= 0; --order)
#pragma unroll
        for (int pb = 0; pb < P; ++pb) {
            const int pa = order - pb;
            if (pa < 0 || pa >= PA) continue;
            if (NT || nb < 2) mma16816(acc, a[0][pa], b[pb][0], b[pb][1]);
            if (!NT || nb >= 2) mma16816(acc, a[1][pa], b[pb][2], b[pb][3]);
        }
}

// The parts of accumulator blocks (2 kk, 2 kk + 1) as a left operand for k block kk.
__device__ __forceinline__ void as_operand(uint32_t (&a)[P][4], const float (&x)[4], const float (&y)[4]) {
    uint32_t o[P];
    split2(x[0], x[1], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][0] = o[p];
    split2(x[2], x[3], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][1] = o[p];
    split2(y[0], y[1], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][2] = o[p];
    split2(y[2], y[3], o);
#pragma unroll
    for (int p = 0; p < P; ++p) a[p][3] = o[p];
}

// A NaN or an infinity of one token must not reach the tokens before it, although a chunk's products meet it with zeros (0 x NaN is
// NaN): where an operand's first parts show one (an infinity also stands for what bf16 cannot hold), such values count as zero, and results
// from the first of a row on are NaN.  The look costs 488 against 470 us (forward, 32 heads of 8192 tokens, d = 128), nothing at d = 64.  (The
// readout takes its product first and again where it has to: looking first, 525 us.)
__device__ __forceinline__ bool not_finite(const uint32_t (&a)[4], const uint32_t (&b)[4]) {
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 z[2] = {zero, zero};                    // 0 x: NaN of what is not finite
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        z[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&a[i]), zero, z[0]);
        z[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&b[i]), zero, z[1]);
    }
    z[0] = __hadd2(z[0], z[1]);
    return __any_sync(~0u, (*reinterpret_cast<uint32_t*>(&z[0]) & 0x7fff7fffu) != 0);
}
// x: a [16 rows x 32 tokens] operand as four blocks of accumulators; first: the first hidden token of rows g and g + 8.
__device__ __forceinline__ void hide_not_finite(float (&x)[4][4], int (&first)[2], int lane) {
    first[0] = first[1] = CT;
#pragma unroll
    for (int nb = 3; nb >= 0; --nb)
#pragma unroll
        for (int q = 3; q >= 0; --q)
            if (__float_as_uint(x[nb][q]) << 1 >= 0x7f7f8000u << 1) {      // what rounds beyond bf16's range
                first[q >> 1] = nb * 8 + 2 * (lane & 3) + (q & 1);
                x[nb][q] = 0.f;
            }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 1; o < 4; o *= 2) first[i] = min(first[i], __shfl_xor_sync(~0u, first[i], o));
}
// Block nb of results: NaN from the first hidden token of each row on.
__device__ __forceinline__ void mark_hidden(float (&x)[4], const int (&first)[2], int nb, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (nb * 8 + 2 * (lane & 3) + (q & 1) >= first[q >> 1]) x[q] = __int_as_float(0x7fffffff);
}

// A token tile in shared memory, as TMA writes it: [part][64-feature half][32 tokens][128 bytes], the 16-byte pieces
// of a row permuted by the row's low bits (128-byte swizzle), so that eight rows' pieces lie in distinct banks.
template <int DK>
constexpr int kTilePart = CT * DK * 2;

// s (16 x DW columns from col0) = fade s + (parts a: 16 x 32 tokens) * X, X a token tile.  Each block's products are
// summed in accumulators of their own, the small ones first, and added to s in fp32.
template <int DK, int DW, int PK>
__device__ __forceinline__ void fade_add_outer(float (&s)[DW / 8][4], float fade, const uint32_t (&a)[2][P][4], uint32_t x, int col0, int lane) {
    const int mi = lane >> 3, lr = lane & 7;
    const int c16 = col0 / 16;                     // first 16-column block: DW / 16 blocks, aligned to their number
    const uint32_t base = x + ((mi & 1) * 8 + lr) * 128 + ((((mi >> 1) ^ lr) << 4) ^ ((c16 & 3) << 5)) + (c16 >> 2) * 4096;
#pragma unroll
    for (int n2 = 0; n2 < DW / 16; ++n2) {
        uint32_t b[2][PK][4];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int pb = 0; pb < PK; ++pb) ldsm4t(b[kk][pb], (base ^ ((n2 & 3) << 5)) + (n2 >> 2) * 4096 + kk * 2048 + pb * kTilePart<DK>);
        float u[2][2][4] = {};
#pragma unroll
        for (int order = P - 1; order >= 0; --order)
#pragma unroll
            for (int pb = 0; pb < PK; ++pb) {
                if (pb > order) continue;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    mma16816(u[kk][0], a[kk][order - pb], b[kk][pb][0], b[kk][pb][1]);
                    mma16816(u[kk][1], a[kk][order - pb], b[kk][pb][2], b[kk][pb][3]);
                }
            }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            s[2 * n2][q] = fmaf(fade, s[2 * n2][q], u[0][0][q] + u[1][0][q]);
            s[2 * n2 + 1][q] = fmaf(fade, s[2 * n2 + 1][q], u[0][1][q] + u[1][1][q]);
        }
    }
}

// acc (16 x 16 tokens, from token 16 n2) += (parts a: 16 x 16 features from col) * X^T, X a token tile: the products of the
// first parts to acc, the others to low.
template <int DK, int PK>
__device__ __forceinline__ void dot_tokens(float (&acc0)[4], float (&acc1)[4], float (&low0)[4], float (&low1)[4], const uint32_t (&a)[P][4],
                                           uint32_t x, int n2, int c16, int lane) {
    const int mi = lane >> 3, lr = lane & 7;
    const uint32_t base = x + (n2 * 16 + (mi >> 1) * 8 + lr) * 128 + ((((mi & 1) ^ lr) << 4) ^ ((c16 & 3) << 5)) + (c16 >> 2) * 4096;
#pragma unroll
    for (int pb = 0; pb < PK; ++pb) {
        uint32_t b[4];
        ldsm4(b, base + pb * kTilePart<DK>);
#pragma unroll
        for (int pa = 0; pa + pb < P; ++pa) {
            mma16816(pa + pb ? low0 : acc0, a[pa], b[0], b[1]);
            mma16816(pa + pb ? low1 : acc1, a[pa], b[2], b[3]);
        }
    }
}

// Byte offset of (row, byte) in a tile of rows of RB bytes (32, 64 or 128) under TMA's swizzle of that width.
template <int RB>
__device__ __forceinline__ uint32_t swz(int row, int byte) {
    const uint32_t o = row * RB + byte;
    return o ^ (((o >> 7) & (RB / 16 - 1)) << 4);
}

__device__ __forceinline__ void sts4(uint32_t a, const float (&v)[4]) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ void sts4u(uint32_t a, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ uint4 lds4u(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
// The sum over a tile's KS warps of one block's partials, in warp order ([warp][4 blocks][32 lanes] float4).
template <int KS>
__device__ __forceinline__ void sum_partials(float (&x)[4], uint32_t buf, int nb, int lane) {
    float4 v = lds4(buf + (nb * 32 + lane) * 16);
#pragma unroll
    for (int k = 1; k < KS; ++k) {
        const float4 w = lds4(buf + ((k * 4 + nb) * 32 + lane) * 16);
        v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
    }
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
// Barrier of the KS warps of tile rt.
template <int KS>
__device__ __forceinline__ void tile_sync(int rt) {
    asm volatile("bar.sync %0, %1;" ::"r"(rt + 1), "n"(KS * 32) : "memory");
}

// Two blocks of 16 rows x 8 tokens (tokens 0 .. 15) -> bf16 rows [token][16] in `stage` (pitch 24) -> global rows.
__device__ __forceinline__ void put_pair(uint32_t stage, const uint32_t (&w)[4], __nv_bfloat16* dst, long long ts, int left, int lane) {
    const int mi = lane >> 3, lr = lane & 7;
    stsm4t(stage + (((mi >> 1) * 8 + lr) * 24 + (mi & 1) * 8) * 2, w[0], w[1], w[2], w[3]);
    __syncwarp();
    const uint4 v = lds4u(stage + (lane >> 1) * 48 + (lane & 1) * 16);
    if ((lane >> 1) < left) *reinterpret_cast<uint4*>(dst + (lane >> 1) * ts + (lane & 1) * 8) = v;
    __syncwarp();
}
// As bf16 parts (x, y: the two blocks' accumulators), each part `ps` elements apart.
__device__ __forceinline__ void put_pair_parts(uint32_t stage, const float (&x)[4], const float (&y)[4], __nv_bfloat16* dst,
                                               long long ps, long long ts, int left, int lane) {
    uint32_t a[P][4];
    as_operand(a, x, y);
#pragma unroll
    for (int p = 0; p < P; ++p) put_pair(stage + p * 16 * 48, a[p], dst + p * ps, ts, left, lane);
}
// As rows of a token tensor (fp32 is written directly: eight lanes hold eight consecutive features, a 32-byte
// sector).
template <int PK>
__device__ __forceinline__ void put_pair_tokens(uint32_t stage, const float (&x)[4], const float (&y)[4], char* base, long long off,
                                                long long ts, int left, int lane) {
    if constexpr (PK == 1) {
        const uint32_t w[4] = {pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(y[0], y[1]), pack2(y[2], y[3])};
        put_pair(stage, w, reinterpret_cast<__nv_bfloat16*>(base) + off, ts, left, lane);
    } else {
        const int g = lane >> 2, t = lane & 3;
        float* o = reinterpret_cast<float*>(base) + off;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int tok = 2 * t + (q & 1);
            if (tok < left) o[tok * ts + g + (q >> 1) * 8] = x[q];
            if (tok + 8 < left) o[(tok + 8) * ts + g + (q >> 1) * 8] = y[q];
        }
    }
}

// A tile's operand parts in shared memory ([k block][part][lane] of 16 bytes) -> its rows [row0, row0 + 16) of the
// state in global memory, bf16 parts [P][dv][DK]; helper `z` of kHelp takes every kHelp-th k block.
template <int DK>
__device__ __forceinline__ void put_state_parts(uint32_t buf, __nv_bfloat16* dst, int dv, int row0, int z, int lane) {
    const int g = lane >> 2, t = lane & 3;
    for (int kk = z; kk < DK / 16; kk += kHelp)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint4 a = lds4u(buf + ((kk * P + p) * 32 + lane) * 16);
            __nv_bfloat16* o = dst + ((long long)p * dv + row0 + g) * DK + kk * 16 + 2 * t;
            *reinterpret_cast<uint32_t*>(o) = a.x;
            *reinterpret_cast<uint32_t*>(o + 8 * DK) = a.y;
            *reinterpret_cast<uint32_t*>(o + 8) = a.z;
            *reinterpret_cast<uint32_t*>(o + 8 * DK + 8) = a.w;
        }
}
template <int DK, int DW>
__device__ __forceinline__ void put_state(const float (&s)[DW / 8][4], float* dst, int row0, int col0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    dst += (long long)(row0 + g) * DK + col0 + 2 * t;
#pragma unroll
    for (int nb = 0; nb < DW / 8; ++nb) {
        *reinterpret_cast<float2*>(dst + nb * 8) = make_float2(s[nb][0], s[nb][1]);
        *reinterpret_cast<float2*>(dst + 8 * DK + nb * 8) = make_float2(s[nb][2], s[nb][3]);
    }
}
template <int DK, int DW>
__device__ __forceinline__ void get_state(float (&s)[DW / 8][4], const float* src, int row0, int col0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nb = 0; nb < DW / 8; ++nb) {
        float2 a = make_float2(0.f, 0.f), b = a;
        if (src) {
            const float* p = src + (long long)(row0 + g) * DK + col0 + 2 * t + nb * 8;
            a = *reinterpret_cast<const float2*>(p);
            b = *reinterpret_cast<const float2*>(p + 8 * DK);
        }
        s[nb][0] = a.x; s[nb][1] = a.y; s[nb][2] = b.x; s[nb][3] = b.y;
    }
}

// A tensor the loading warp takes tiles of: its tensor map (5-D: features, tokens, heads, images, parts; a box is
// 32 tokens of up to 128 bytes), and the plain view behind it.  A broadcast dimension has extent one in the map.
struct Tiled {
    CUtensorMap map;
    const char* p;
    long long ps, bs, hs, ts;         // strides in elements
    int hmul, bmul;                   // 0 where the dimension is broadcast
    int tma;                          // the map is valid
};

// The loading warp's side of one stage.  Whole chunks come as TMA boxes.  The last, partial chunk of a sequence is
// copied by the warp itself: rows past the end repeat the last token's (they have a step size of zero and are
// never written out, so any finite values do; what lies behind the sequence in memory is not read).
struct Loader {
    uint64_t* bar;
    int lane;
    __device__ __forceinline__ void flat(uint32_t dst, const uint8_t* src, uint32_t bytes) const {
        if (lane == 0)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                         "r"(bytes), "r"(s32(bar))
                         : "memory");
    }
    // features [col, col + RB / E) of one part of 32 tokens, as a swizzled tile of rows of RB bytes
    template <int RB, int E>
    __device__ __forceinline__ void tile(uint32_t dst, const Tiled& x, int part, int b, int head, int tok, int col, int left) const {
        if (x.tma && left >= CT) {
            if (lane == 0)
                asm volatile(
                    "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
                    "[%2];" ::"r"(dst),
                    "l"(&x.map), "r"(s32(bar)), "r"(col), "r"(tok), "r"(head * x.hmul), "r"(b * x.bmul), "r"(part)
                    : "memory");
            return;
        }
        constexpr int CPR = RB / 16;
        const char* src = x.p + (part * x.ps + b * x.bs + head * x.hs + tok * x.ts + col) * E;
        uint4 v[CPR];
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
            const int row = (i * 32 + lane) / CPR, c = (i * 32 + lane) % CPR;
            v[i] = *reinterpret_cast<const uint4*>(src + min(row, left - 1) * x.ts * E + c * 16);
        }
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
            const int row = (i * 32 + lane) / CPR, c = (i * 32 + lane) % CPR;
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + swz<RB>(row, c * 16)), "r"(v[i].x), "r"(v[i].y),
                         "r"(v[i].z), "r"(v[i].w)
                         : "memory");
        }
    }
    // bytes of a tile that arrive by TMA
    __device__ __forceinline__ static uint32_t bytes(const Tiled& x, int left, uint32_t n) { return x.tma && left >= CT ? n : 0; }
};
template <int DK, int PK>
__device__ __forceinline__ void load_tokens(const Loader& l, uint32_t dst, const Tiled& x, int b, int head, int tok, int left) {
#pragma unroll
    for (int p = 0; p < PK; ++p)
#pragma unroll
        for (int c = 0; c < DK; c += 64) l.template tile<128, 2>(dst + p * kTilePart<DK> + c / 64 * 4096, x, p, b, head, tok, c, left);
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

// Periods c = 0 .. chunks.  In period c the chain warps take chunk c from the state they hold to the next one
// and leave the state they started from (as operand parts) and the residuals E in shared memory; the helpers finish
// chunk c - 1 from those: its readout (forward), or E and the state to global memory (backward, SAVE);
// the loading warp is one or two periods ahead.
template <int DK, int PK, int RT, int KS, bool SAVE>
__device__ __forceinline__ void chain_body(const Dims& d, const Tiled& Q, const Tiled& K, const Tiled& V, const uint8_t* rec, const float* W0,
                                           long long w0_bs, const ChainOut& out, uint32_t* err, unsigned long long wait_ns, int block) {
    using L = ChainLayout<DK, PK, RT, KS, SAVE>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (s32(smem_raw) & 1023));
    constexpr int DW = DK / KS, KB = DW / 16, NBW = 4 / KS, CW = RT * KS, HW = RT * kHelp;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int slices = d.dv / L::VW;
    const int slice = block % slices;
    const int bh = block / slices, b = bh / d.h, h = bh % d.h;
    pdl_wait_primary();
    const int len = seq_len(d, b), nch = (len + CT - 1) / CT;
    const int v0 = slice * L::VW;
    const long long state = (long long)d.dv * DK;
    const uint32_t sb = s32(smem), gates = sb + L::kStages * L::stage;
    const uint32_t sbuf = gates + L::kGates, ebuf = sbuf + 2 * RT * L::kS, xbuf = ebuf + 2 * RT * L::kE, obuf = xbuf + L::kX;
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem + L::smem - 1024 - kCtlBytes);
    auto gate_slot = [&](int c) { return gates + (c & (kGateSlots - 1)) * kGateBytes; };
    auto stage_of = [&](int c) { return sb + (c % L::kStages) * L::stage; };

    if (warp == CW + HW) {
        // ---------------------------------------------------------------- loads
        const int recb = rec_bytes(SAVE);
        const Abort ab{&ctl.abort_flag, err, wait_ns};
        if (lane == 0) {
            ctl.abort_flag = 0;
            for (int i = 0; i < L::kStages; ++i) mbar_init(&ctl.full[i], 1);
            fence_barrier_init();
        }
        __syncwarp();
        auto loads_in = [&](int c) { return c < nch || (!SAVE && c == nch && nch > 0); };
        auto issue = [&](int c) {
            if (!loads_in(c)) return;
            const uint32_t st = stage_of(c);
            const uint8_t* r = rec + ((long long)bh * d.nc + c) * recb;
            const Loader l{&ctl.full[c % L::kStages], lane};
            const bool now = c < nch, before = !SAVE && c >= 1;
            const int left = len - c * CT;
            if (lane == 0) {
                fence_proxy_async_smem();             // the warp's own stores to the stage, before the copies' writes
                uint32_t n = 0;
                if (now) n += Loader::bytes(K, left, L::kK) + Loader::bytes(V, left, L::kV) + kGateBytes + L::kT;
                if (before) n += Loader::bytes(Q, left + CT, L::kK) + L::kA;
                mbar_arrive_expect_tx(l.bar, n);
            }
            __syncwarp();
            if (now) {
                load_tokens<DK, PK>(l, st, K, b, h / d.r, c * CT, left);
                l.template tile<L::VB, PK == 1 ? 2 : 4>(st + L::kK + L::kQ, V, 0, b, h, c * CT, v0, left);
                l.flat(gate_slot(c), r, kGateBytes);
                l.flat(st + L::kK + L::kQ + L::kV, r + kGateBytes, L::kT);
            }
            if (before) {
                load_tokens<DK, PK>(l, st + L::kK, Q, b, h / d.r, c * CT - CT, left + CT);
                l.flat(st + L::kK + L::kQ + L::kV + L::kT, r - recb + kGateBytes + kMat, L::kA);
            }
        };
        for (int c = 0; c < L::kStages - 1; ++c) issue(c);
        int good = nch + 1;                           // periods before the first whose loads did not come in time
        for (int c = 0; c <= nch; ++c) {
            if (c < good && loads_in(c) && !__all_sync(~0u, mbar_wait(&ctl.full[c % L::kStages], (c / L::kStages) & 1, ab))) good = c;
            __syncthreads();
            if (c < good) issue(c + L::kStages - 1);
        }
        for (int c = good; c <= nch && c < good + L::kStages - 1; ++c)       // nothing may still be on its way when the CTA ends
            if (loads_in(c)) mbar_drain(&ctl.full[c % L::kStages], (c / L::kStages) & 1, drain_limit(ab));
        return;
    }
    if (warp >= CW) {
        // ---------------------------------------------------------------- helpers
        const int hw = warp - CW, rt = hw % RT, z = hw / RT, row0 = v0 + rt * 16;
        const uint32_t stagebuf = obuf + hw * P * 16 * 48;
        for (int c = 0; c <= nch; ++c) {
            __syncthreads();
            if (c == 0) continue;
            const int pc = c - 1, left = len - pc * CT;
            const uint32_t sp = sbuf + ((pc & 1) * RT + rt) * L::kS, ep = ebuf + ((pc & 1) * RT + rt) * L::kE, gt = gate_slot(pc);
            if constexpr (SAVE) {
                const float4 v = lds4(ep + (2 * z * 32 + lane) * 16), w = lds4(ep + ((2 * z + 1) * 32 + lane) * 16);
                const float e0[4] = {v.x, v.y, v.z, v.w}, e1[4] = {w.x, w.y, w.z, w.w};
                put_pair_parts(stagebuf, e0, e1, out.E + ((long long)bh * d.N + (long long)pc * CT + z * 16) * d.dv + row0, out.e_ps,
                                  d.dv, left - z * 16, lane);
                if ((pc * CT) % d.gt == 0)
                    put_state_parts<DK>(sp, out.S + ((long long)bh * d.ng + (pc * CT) / d.gt) * P * state, d.dv, row0, z, lane);
            } else {
                // Z of tokens [16 z, 16 z + 16) = scale gamma (Q W^T) + A U
                const uint32_t st = stage_of(c), qt = st + L::kK, am = st + L::kK + L::kQ + L::kV + L::kT;
                float acc[2][4] = {}, low[2][4] = {};
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk) {
                    uint32_t a[P][4];
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const uint4 v = lds4u(sp + ((kk * P + p) * 32 + lane) * 16);
                        a[p][0] = v.x; a[p][1] = v.y; a[p][2] = v.z; a[p][3] = v.w;
                    }
                    dot_tokens<DK, PK>(acc[0], acc[1], low[0], low[1], a, qt, z, kk, lane);
                }
                float e[4][4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) {
                    const float4 v = lds4(ep + (nb * 32 + lane) * 16);
                    const float2 be = lds2(gt + (2 * CT + nb * 8 + 2 * t) * 4);
                    e[nb][0] = be.x * v.x; e[nb][1] = be.y * v.y; e[nb][2] = be.x * v.z; e[nb][3] = be.y * v.w;
                }
                uint32_t u[2][P][4];
                as_operand(u[0], e[0], e[1]);
                as_operand(u[1], e[2], e[3]);
                float au[2][4] = {};
#pragma unroll
                for (int i = 0; i < 2; ++i) mat_block<P, true>(au[i], u, am, 2 * z + i, lane);
                if (not_finite(u[0][0], u[1][0])) {
                    int first[2];
                    hide_not_finite(e, first, lane);
                    as_operand(u[0], e[0], e[1]);
                    as_operand(u[1], e[2], e[3]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        au[i][0] = au[i][1] = au[i][2] = au[i][3] = 0.f;
                        mat_block<P, true>(au[i], u, am, 2 * z + i, lane);
                        mark_hidden(au[i], first, 2 * z + i, lane);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int nb = 2 * z + i;
                    const float2 ga = lds2(gt + (nb * 8 + 2 * t) * 4);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(d.scale * ((q & 1) ? ga.y : ga.x), acc[i][q] + low[i][q], au[i][q]);
                }
                put_pair_tokens<PK>(stagebuf, acc[0], acc[1], out.Z.p,
                                    b * out.Z.bs + h * out.Z.hs + ((long long)pc * CT + z * 16) * out.Z.ts + row0, out.Z.ts, left - z * 16, lane);
            }
        }
        return;
    }
    // -------------------------------------------------------------------- chain
    const int ks = warp % KS, rt = warp / KS, col0 = ks * DW, row0 = v0 + rt * 16;
    const uint32_t xp = xbuf + rt * KS * L::kE;
    float s[DW / 8][4];
    get_state<DK, DW>(s, W0 ? W0 + b * w0_bs + h * state : nullptr, row0, col0, lane);
    for (int c = 0; c <= nch; ++c) {
        __syncthreads();
        if (c == nch) break;
        const uint32_t st = stage_of(c), kt = st, vt = st + L::kK + L::kQ, tm = vt + L::kV, gt = gate_slot(c);
        const uint32_t sp = sbuf + ((c & 1) * RT + rt) * L::kS, ep = ebuf + ((c & 1) * RT + rt) * L::kE;
        const bool hand = !SAVE || (c * CT) % d.gt == 0;

        float x[4][4] = {}, low[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
            uint32_t a[P][4];
            as_operand(a, s[2 * kk], s[2 * kk + 1]);
#pragma unroll
            for (int n2 = 0; n2 < 2; ++n2)
                dot_tokens<DK, PK>(x[2 * n2], x[2 * n2 + 1], low[2 * n2], low[2 * n2 + 1], a, kt, n2, ks * KB + kk, lane);
            if (hand) {
#pragma unroll
                for (int p = 0; p < P; ++p) sts4u(sp + (((ks * KB + kk) * P + p) * 32 + lane) * 16, a[p]);
            }
        }
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) x[nb][q] += low[nb][q];
        if constexpr (KS > 1) {
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) sts4(xp + ((ks * 4 + nb) * 32 + lane) * 16, x[nb]);
            tile_sync<KS>(rt);
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) sum_partials<KS>(x[nb], xp, nb, lane);
        }
        // R = V - gamma (W K^T)
#pragma unroll
        for (int n2 = 0; n2 < 2; ++n2) {
            float v[2][4];
            if constexpr (PK == 1) {
                uint32_t r[4];
                const int mi = lane >> 3, lr = lane & 7;
                ldsm4t(r, vt + swz<L::VB>(n2 * 16 + (mi >> 1) * 8 + lr, rt * 32 + (mi & 1) * 16));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i >> 1][2 * (i & 1)] = lo_f(r[i]);
                    v[i >> 1][2 * (i & 1) + 1] = hi_f(r[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[i][q] = lds1(vt + swz<L::VB>(n2 * 16 + i * 8 + 2 * t + (q & 1), (rt * 16 + g + (q >> 1) * 8) * 4));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int nb = 2 * n2 + i;
                const float2 ga = lds2(gt + (nb * 8 + 2 * t) * 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) x[nb][q] = fmaf(-((q & 1) ? ga.y : ga.x), x[nb][q], v[i][q]);
            }
        }
        // E = T' R
        float e[4][4] = {};
        uint32_t a[2][P][4];
        as_operand(a[0], x[0], x[1]);
        as_operand(a[1], x[2], x[3]);
        int first[2];
        const bool hidden = not_finite(a[0][0], a[1][0]);
        if (hidden) {
            hide_not_finite(x, first, lane);
            as_operand(a[0], x[0], x[1]);
            as_operand(a[1], x[2], x[3]);
        }
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) mat_block<P, true>(e[nb], a, tm, nb, lane);
        if (hidden)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) mark_hidden(e[nb], first, nb, lane);
        // W <- gamma_C W + (suffix beta E)^T K
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            if (nb / NBW == ks) sts4(ep + (nb * 32 + lane) * 16, e[nb]);
            const float2 su = lds2(gt + (CT + nb * 8 + 2 * t) * 4), be = lds2(gt + (2 * CT + nb * 8 + 2 * t) * 4);
            const float u0 = su.x * be.x, u1 = su.y * be.y;
            e[nb][0] *= u0; e[nb][1] *= u1; e[nb][2] *= u0; e[nb][3] *= u1;
        }
        as_operand(a[0], e[0], e[1]);
        as_operand(a[1], e[2], e[3]);
        fade_add_outer<DK, DW, PK>(s, lds1(gt + (CT - 1) * 4), a, kt, col0, lane);
    }
    if (out.W1) put_state<DK, DW>(s, out.W1 + (long long)bh * state, row0, col0, lane);
}

struct ChainArgs {
    Dims d;
    Tiled Q, K, V;
    const uint8_t* rec;
    const float* W0;
    long long w0_bs;
    ChainOut out;
    uint32_t* err;
    unsigned long long wait_ns;
};
template <int DK, int PK, int RT, int KS>
__global__ void __launch_bounds__(seq_warps<RT, KS>() * 32)
delta_chain(const __grid_constant__ ChainArgs a) {
    pdl_launch_dependents();
    chain_body<DK, PK, RT, KS, false>(a.d, a.Q, a.K, a.V, a.rec, a.W0, a.w0_bs, a.out, a.err, a.wait_ns, blockIdx.x);
}

// A five-dimensional tensor map: boxes of `rows` along the second dimension x rb bytes (32, 64 or 128, swizzled alike)
// along the first.  strides: elements, of dimensions 1 .. 4.
static bool encode_map(CUtensorMap* m, const void* p, int esz, std::array<cuuint64_t, 5> dims, std::array<long long, 4> strides, int rb,
                       int rows) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                               CUtensorMapFloatOOBfill);
    static const Encode enc = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<Encode>(f) : nullptr;
    }();
    if (!enc) return false;
    cuuint64_t bytes[4];
    for (int i = 0; i < 4; ++i) {
        bytes[i] = (cuuint64_t)strides[i] * esz;
        if (bytes[i] >= (1ull << 40)) return false;
    }
    const cuuint32_t box[5] = {(cuuint32_t)(rb / esz), (cuuint32_t)rows, 1, 1, 1}, one[5] = {1, 1, 1, 1, 1};
    return enc(m, esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 5, const_cast<void*>(p), dims.data(),
               bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The map of a [part][batch][heads][tokens][width] tensor with boxes of 32 tokens x rb bytes.
static Tiled tiled(const void* p, long long ps, int parts, long long bs, long long hs, long long ts, const Dims& d, int heads, int width,
                   int esz, int rb) {
    Tiled x{};
    x.p = static_cast<const char*>(p);
    x.ps = ps; x.bs = bs; x.hs = hs; x.ts = ts;
    x.hmul = hs != 0;
    x.bmul = bs != 0;
    // a dimension of size one keeps a stride that is valid
    x.tma = (ts != 0 || d.N == 1) &&
            encode_map(&x.map, p, esz, {(cuuint64_t)width, (cuuint64_t)d.N, (cuuint64_t)(hs ? heads : 1), (cuuint64_t)(bs ? d.B : 1), (cuuint64_t)parts},
                       {ts ? ts : width, hs ? hs : width, bs ? bs : width, ps ? ps : width}, rb, CT);
    return x;
}
static Tiled tiled(const Parts& x, int parts, const Dims& d, int heads, int width, int rb) {
    return tiled(x.p, x.ps, parts, x.bs, x.hs, x.ts, d, heads, width, 2, rb);
}

// Launches `k` as a programmatic dependent of what precedes it in the stream: its set-up overlaps that kernel's tail.
// (Every kernel here waits for its predecessor before it reads or writes global memory.  split_tokens and the step are plain launches.)
template <class... T, class... A>
static ttt_status launch(void (*k)(T...), long long grid, int threads, int smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return check_launch(cudaLaunchKernelEx(&cfg, k, T(args)...));
}

// Shared memory that leaves room for no second CTA of the same kernel on an SM: a grid that fits the SMs is spread over
// them even while the kernel before it still holds some (two on one SM take longer than two side by side).
constexpr int kAloneSmem = 116 * 1024;
static int spread_smem(int smem, long long grid, int sms) { return grid <= sms && smem < kAloneSmem ? kAloneSmem : smem; }

// Lets `kernel` use `bytes` of dynamic shared memory on the current device (set once per kernel and device).
template <auto kernel>
static ttt_status allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};            // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return check_launch(e);
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return TTT_OK;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return check_launch(e);
}

static uint32_t* error_word(const Call& c) { return reinterpret_cast<uint32_t*>(c.ws); }

#include "delta_backward.cuh"

// --------------------------------------------------------------------------------------------------
// Workspace
// --------------------------------------------------------------------------------------------------
struct Layout {
    size_t rec, qp, kp, op, E, Y, S, D, dw, part, total;
};
static Layout layout(const Dims& d, bool fp32, bool backward) {
    Layout l{};
    size_t at = kWsHeader;
    auto take = [&](size_t bytes) { const size_t o = at; at = align_up(at + bytes, 256); return o; };
    const size_t heads = (size_t)d.B * d.h, toks = heads * d.N;
    l.rec = take(heads * d.nc * rec_bytes(backward));
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
        if (d.r > 1) l.part = take(2 * toks * d.dk * 4);
    }
    l.total = at;
    return l;
}
size_t forward_ws_bytes(const Dims& d, bool fp32) { return layout(d, fp32, false).total; }
size_t backward_ws_bytes(const Dims& d, bool fp32) { return layout(d, fp32, true).total; }

// --------------------------------------------------------------------------------------------------
// Launches
// --------------------------------------------------------------------------------------------------

// Token tensors as bf16 parts: themselves (bf16), or 3 parts each in the workspace (fp32; one launch for all).
struct Splitter {
    const Call& c;
    bool fp32;
    SplitArgs a{};
    int n = 0;
    Parts add(const View& x, uint8_t* ws, int heads, int width) {
        if (!fp32) return Parts{reinterpret_cast<const __nv_bfloat16*>(x.p), 0, x.bs, x.hs, x.ts};
        const long long ps = (long long)c.d.B * heads * c.d.N * width;
        a.x[n] = x;
        a.out[n] = reinterpret_cast<__nv_bfloat16*>(ws);
        a.ps[n] = ps;
        a.heads[n] = heads;
        a.width[n++] = width;
        return Parts{reinterpret_cast<__nv_bfloat16*>(ws), ps, (long long)heads * c.d.N * width, (long long)c.d.N * width, width};
    }
    ttt_status run() {
        if (!n) return TTT_OK;
        a.d = c.d;
        long long most = 0;
        for (int i = 0; i < n; ++i) most = std::max(most, a.ps[i]);
        split_tokens<<<dim3((unsigned)std::min<long long>((most / 4 + 255) / 256, 8LL * c.sms), n), 256, 0, c.stream>>>(a);
        return check_launch(cudaGetLastError());
    }
};

template <int DK, int PK, bool BACKWARD>
static ttt_status run_prep(const Call& c, const Parts& Q, const Parts& K, uint8_t* rec) {
    constexpr int smem = kPrepWarps * kPrepWarpBytes;
    constexpr auto k = delta_prep<DK, PK, BACKWARD>;
    ttt_status st = allow_smem<k>(smem);
    if (st != TTT_OK) return st;
    const long long total = (long long)c.d.B * c.d.h * c.d.nc;
    return launch(k, (total + kPrepWarps - 1) / kPrepWarps, kPrepWarps * 32, smem, c.stream, c.d, Q, K, c.G, c.Beta, rec, total, error_word(c));
}

template <int DK, int PK, int RT, int KS>
static ttt_status run_chain_t(const Call& c, const Parts& Q, const Parts& K, const uint8_t* rec, const ChainOut& out) {
    using L = ChainLayout<DK, PK, RT, KS, false>;
    static_assert(L::smem <= 227 * 1024, "shared memory of a chain CTA");
    constexpr auto k = delta_chain<DK, PK, RT, KS>;
    const ttt_status st = allow_smem<k>(std::max(L::smem, kAloneSmem));
    if (st != TTT_OK) return st;
    const long long grid = (long long)c.d.B * c.d.h * (c.d.dv / L::VW);
    const ChainArgs a{c.d, tiled(Q, PK, c.d, c.d.hk, DK, 128), tiled(K, PK, c.d, c.d.hk, DK, 128),
                      tiled(c.V.p, 0, 1, c.V.bs, c.V.hs, c.V.ts, c.d, c.d.h, c.d.dv, PK == 1 ? 2 : 4, L::VB), rec, c.W0, c.w0_bs, out,
                      error_word(c), c.wait_ns};
    return launch(k, grid, seq_warps<RT, KS>() * 32, spread_smem(L::smem, grid, c.sms), c.stream, a);
}

template <int DK, int PK>
static ttt_status forward_t(const Call& c) {
    const Layout l = layout(c.d, PK == 3, false);
    Splitter split{c, PK == 3};
    const Parts Q = split.add(c.Q, c.ws + l.qp, c.d.hk, DK), K = split.add(c.K, c.ws + l.kp, c.d.hk, DK);
    ttt_status st = split.run();
    if (st == TTT_OK) st = run_prep<DK, PK, false>(c, Q, K, c.ws + l.rec);
    if (st != TTT_OK) return st;
    ChainOut out{};
    out.Z = c.Z;
    out.W1 = c.W1_out;
    return few_tiles(c, 1) ? run_chain_t<DK, PK, 1, 2>(c, Q, K, c.ws + l.rec, out) : run_chain_t<DK, PK, 2, 2>(c, Q, K, c.ws + l.rec, out);
}

template <int DK, int PK>
static ttt_status backward_t(const Call& c) {
    constexpr bool F = PK == 3;
    const Layout l = layout(c.d, F, true);
    uint8_t* rec = c.ws + l.rec;
    const long long ps = (long long)c.d.B * c.d.h * c.d.N * c.d.dv;
    ChainOut out{};
    out.E = reinterpret_cast<__nv_bfloat16*>(c.ws + l.E);
    out.e_ps = ps;
    out.S = reinterpret_cast<__nv_bfloat16*>(c.ws + l.S);
    BackOut bo{};
    bo.dV = c.dV;
    bo.Y = reinterpret_cast<__nv_bfloat16*>(c.ws + l.Y);
    bo.y_ps = ps;
    bo.D = reinterpret_cast<__nv_bfloat16*>(c.ws + l.D);
    const bool reduce = c.dW0 && c.w0_bs == 0;
    bo.dW0 = reduce ? reinterpret_cast<float*>(c.ws + l.dw) : c.dW0;
    Splitter split{c, F};
    const Parts Q = split.add(c.Q, c.ws + l.qp, c.d.hk, DK), K = split.add(c.K, c.ws + l.kp, c.d.hk, DK),
                O = split.add(c.Z, c.ws + l.op, c.d.h, c.d.dv);
    ttt_status st = split.run();
    if (st != TTT_OK) return st;
    st = run_prep<DK, PK, true>(c, Q, K, rec);
    if (st == TTT_OK) st = run_both<DK, PK>(c, Q, K, O, rec, out, bo);
    if (st == TTT_OK) st = run_grads<DK, PK>(c, Q, K, O, out, bo, reinterpret_cast<float*>(c.ws + l.part));
    if (st != TTT_OK || !reduce) return st;
    return run_sum_images(bo.dW0, c.dW0, c.d.B, (long long)c.d.h * c.d.dv * DK, c.stream);
}

ttt_status launch_forward(const Call& c) {
    if (c.fp32) return c.d.dk == 64 ? forward_t<64, 3>(c) : forward_t<128, 3>(c);
    return c.d.dk == 64 ? forward_t<64, 1>(c) : forward_t<128, 1>(c);
}
ttt_status launch_backward(const Call& c) {
    if (c.fp32) return c.d.dk == 64 ? backward_t<64, 3>(c) : backward_t<128, 3>(c);
    return c.d.dk == 64 ? backward_t<64, 1>(c) : backward_t<128, 1>(c);
}

}  // namespace gd
}  // namespace ttt
