// delta_backward.cuh -- backward pass of the gated delta rule (included by delta.cu, inside ttt::gd).
//
// With D the adjoint of the state, y_t = D_t k_t that of the update u_t = beta_t e_t, and dz' = scale dz:
//   reverse (one warp per 16 rows of D, sequential from the last chunk to the first):
//     dU = diag(Gamma_C.) K D^T + A^T dZ,   Y = T_u^T dU  with T_u = (I + diag(beta) G)^{-1},
//     dV = diag(beta) Y,   D <- gamma_C D + (diag(gamma) dZ')^T Q - (diag(gamma) dV)^T K;
//   grads (one CTA per image, key head and group of tokens, all at once), from E, Y (per token), W at the
//     group's start and D at its end, with the group's own gamma and Gamma:
//     H_ij = scale Gamma_ij beta_j dz_i.e_j (j <= i),   F_ij = -beta_i beta_j Gamma_ij y_i.e_j (j < i),
//     dQ_i = scale gamma_i W^T dz_i + sum_j H_ij k_j,
//     dK_i = beta_i Gamma_Ci D^T e_i - gamma_i beta_i W^T y_i + sum_j F_ij k_j + sum_j (H_ji q_j + F_ji k_j),
//     dbeta_i = y_i.e_i,
//     dg_l = gamma_C <D, W> + sum_{j<l} k_j.(first term of dK_j)
//            + sum_{i>=l} (q_i.dQ_i + k_i.(second and third terms of dK_i) - k_i.(last term of dK_i)).
//   E and W come from the forward chain run again (they are not kept from the forward call).
// All products take P bf16 parts per inexact operand, as the forward pass.

struct BackOut {
    View dV;
    __nv_bfloat16* Y;             // [P][B][h][N][dv]
    long long y_ps;
    __nv_bfloat16* D;             // adjoints at the groups' ends [B][h][ng][P][dv][dk]
    float* dW0;                   // nullable [B][h][dv][dk]
};

// As mat_nt with the image's rows along k: acc[n = column j] += a (k = row i) * M[i][j], i >= j blocks only.
template <int P, int PA>
__device__ __forceinline__ void mat_nn(float (&acc)[4][4], const uint32_t (&a)[PA][4], uint32_t mat, int kk, int lane) {
    const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
    for (int n2 = 0; n2 <= kk; ++n2)
#pragma unroll
        for (int pb = 0; pb < P; ++pb) {
            uint32_t b[4];
            ldsm4t(b, mat + ((pb * CT + kk * 16 + (mi & 1) * 8 + lr) * MP + n2 * 16 + (mi >> 1) * 8) * 2);
#pragma unroll
            for (int pa = 0; pa < PA; ++pa)
                if (pa + pb < P) {
                    mma16816(acc[2 * n2], a[pa], b[0], b[1]);
                    mma16816(acc[2 * n2 + 1], a[pa], b[2], b[3]);
                }
        }
}

template <int DK, int P, int PK, int NW>
struct ReverseLayout {
    static constexpr int KP = DK + 8, VW = NW * 16, VP = VW + 8;
    static constexpr int kK = PK * CT * KP * 2;
    static constexpr int kO = PK * CT * VP * 2;
    static constexpr int kR = kGateBytes + 2 * mat_bytes(P);
    static constexpr int stage = 2 * kK + kO + kR;
    static constexpr int kStages = 3 * stage <= 110 * 1024 ? 3 : 2;
    static constexpr int warp_out = CT * 24 * 2;
    static constexpr int smem = kStages * stage + NW * warp_out;
};

template <int DK, int P, int PK, int NW>
__global__ void __launch_bounds__(NW * 32)
delta_reverse(Dims d, Parts Q, Parts K, Parts O, const uint8_t* rec, const float* dW1, BackOut out) {
    using L = ReverseLayout<DK, P, PK, NW>;
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int NT = NW * 32, KP = L::KP;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3;
    const int slices = d.dv / L::VW;
    const int slice = blockIdx.x % slices;
    const int bh = blockIdx.x / slices, b = bh / d.h, h = bh % d.h;
    const int len = seq_len(d, b), nch = (len + CT - 1) / CT;
    const int v0 = slice * L::VW, row0 = v0 + warp * 16;
    const uint32_t sb = s32(smem), wout = sb + L::kStages * L::stage + warp * L::warp_out;
    const int recb = rec_bytes(P, true);

    auto issue = [&](int k) {                     // k-th chunk from the end
        const int c = nch - 1 - k;
        if (c >= 0) {
            const uint32_t st = sb + (k % L::kStages) * L::stage;
            const int left = len - c * CT;
            const long long tok = (long long)c * CT;
#pragma unroll
            for (int p = 0; p < PK; ++p) {
                load_rows<DK, 2, NT>(st + p * CT * KP * 2, KP * 2,
                                     reinterpret_cast<const char*>(K.p + p * K.ps + b * K.bs + (h / d.r) * K.hs + tok * K.ts),
                                     K.ts * 2, left, tid);
                load_rows<DK, 2, NT>(st + L::kK + p * CT * KP * 2, KP * 2,
                                     reinterpret_cast<const char*>(Q.p + p * Q.ps + b * Q.bs + (h / d.r) * Q.hs + tok * Q.ts),
                                     Q.ts * 2, left, tid);
                load_rows<L::VW, 2, NT>(st + 2 * L::kK + p * CT * L::VP * 2, L::VP * 2,
                                        reinterpret_cast<const char*>(O.p + p * O.ps + b * O.bs + h * O.hs + tok * O.ts + v0),
                                        O.ts * 2, left, tid);
            }
            const uint8_t* r = rec + ((long long)bh * d.nc + c) * recb;
            load_flat<kGateBytes, NT>(st + 2 * L::kK + L::kO, r, tid);
            load_flat<2 * mat_bytes(P), NT>(st + 2 * L::kK + L::kO + kGateBytes, r + kGateBytes + mat_bytes(P), tid);
        }
        cp_commit();
    };

    float s[DK / 8][4];
    const long long state = (long long)d.dv * DK;
    get_state<DK>(s, dW1 ? dW1 + bh * state : nullptr, row0, lane);
    for (int k = 0; k < L::kStages - 1; ++k) issue(k);

    for (int k = 0; k < nch; ++k) {
        const int c = nch - 1 - k;
        cp_wait<L::kStages - 2>();
        __syncthreads();
        issue(k + L::kStages - 1);
        const uint32_t st = sb + (k % L::kStages) * L::stage;
        const uint32_t kt = st, qt = st + L::kK, ot = st + 2 * L::kK, gt = ot + L::kO, am = gt + kGateBytes, um = am + mat_bytes(P);
        const int left = len - c * CT;
        if (k == 0 || ((c + 1) * CT) % d.gt == 0)
            put_state_parts<DK, P>(s, out.D + ((long long)bh * d.ng + (c * CT) / d.gt) * P * state, d.dv, row0, lane);

        float x[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
            uint32_t a[P][4];
            as_operand<P>(a, s[2 * kk], s[2 * kk + 1]);
            dot_tokens<DK, P, PK>(x, a, kt, kk, lane);
        }
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float2 su = lds2(gt + (CT + nb * 8 + 2 * t) * 4);
            x[nb][0] *= su.x; x[nb][1] *= su.y; x[nb][2] *= su.x; x[nb][3] *= su.y;
        }
        // dU += dZ^T A;   the scaled dZ' as the left operand of the state's update
        const float gc = lds1(gt + (CT - 1) * 4);
#pragma unroll
        for (int nb = 0; nb < DK / 8; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) s[nb][q] *= gc;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t o[PK][4];
            const int mi = lane >> 3, lr = lane & 7;
#pragma unroll
            for (int p = 0; p < PK; ++p)
                ldsm4t(o[p], ot + ((p * CT + kk * 16 + (mi >> 1) * 8 + lr) * L::VP + warp * 16 + (mi & 1) * 8) * 2);
            mat_nn<P, PK>(x, o, am, kk, lane);
            float f[2][4];                        // tokens kk 16 + 2t (+1), then + 8
            const float2 g0 = lds2(gt + (kk * 16 + 2 * t) * 4), g1 = lds2(gt + (kk * 16 + 8 + 2 * t) * 4);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f[0][2 * q] = lo_f(o[0][q]);
                f[0][2 * q + 1] = hi_f(o[0][q]);
                f[1][2 * q] = lo_f(o[0][2 + q]);
                f[1][2 * q + 1] = hi_f(o[0][2 + q]);
#pragma unroll
                for (int p = 1; p < PK; ++p) {
                    f[0][2 * q] += lo_f(o[p][q]);
                    f[0][2 * q + 1] += hi_f(o[p][q]);
                    f[1][2 * q] += lo_f(o[p][2 + q]);
                    f[1][2 * q + 1] += hi_f(o[p][2 + q]);
                }
                f[0][2 * q] *= d.scale * g0.x;
                f[0][2 * q + 1] *= d.scale * g0.y;
                f[1][2 * q] *= d.scale * g1.x;
                f[1][2 * q + 1] *= d.scale * g1.y;
            }
            uint32_t a[P][4];
            as_operand<P>(a, f[0], f[1]);
            add_outer<DK, P, PK>(s, a, qt, kk, lane);
        }
        // Y = T_u^T dU
        float y[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t a[P][4];
            as_operand<P>(a, x[2 * kk], x[2 * kk + 1]);
            mat_nn<P, P>(y, a, um, kk, lane);
        }
        put_rows_parts<P>(wout, y, out.Y + ((long long)bh * d.N + (long long)c * CT) * d.dv + row0, out.y_ps, d.dv, left, lane);
        // dV = beta Y;   D -= (gamma dV)^T K
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float2 be = lds2(gt + (2 * CT + nb * 8 + 2 * t) * 4);
            y[nb][0] *= be.x; y[nb][1] *= be.y; y[nb][2] *= be.x; y[nb][3] *= be.y;
        }
        put_tokens<PK>(wout, y, out.dV.p, b * out.dV.bs + h * out.dV.hs + (long long)c * CT * out.dV.ts + row0, out.dV.ts, left, lane);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float2 ga = lds2(gt + (nb * 8 + 2 * t) * 4);
            y[nb][0] *= -ga.x; y[nb][1] *= -ga.y; y[nb][2] *= -ga.x; y[nb][3] *= -ga.y;
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t a[P][4];
            as_operand<P>(a, y[2 * kk], y[2 * kk + 1]);
            add_outer<DK, P, PK>(s, a, kt, kk, lane);
        }
    }
    cp_wait<0>();
    if (out.dW0) put_state<DK>(s, out.dW0 + bh * state, row0, lane);
}

// --------------------------------------------------------------------------------------------------
// Token gradients
// --------------------------------------------------------------------------------------------------
template <int DK, int P, int PK>
struct GradsLayout {
    static constexpr int GT = PK == 3 ? 32 : 64;                // tokens per group
    static constexpr int SV = 32;                               // value features per slice
    static constexpr int KP = DK + 8, SP = SV + 8, HP = GT + 8, FP = GT + 1;
    static constexpr int kK = PK * GT * KP * 2;                 // K, and Q
    static constexpr int kO = PK * GT * SP * 2;
    static constexpr int kE = P * GT * SP * 2;                  // E, and Y
    static constexpr int kS = P * SV * KP * 2;                  // W, and D
    static constexpr int stage = kO + 2 * kE + 2 * kS;
    static constexpr int kH = P * GT * HP * 2;                  // H, and F: in the stages' memory after the slices
    static_assert(2 * kH <= 2 * stage, "H and F fit the stages");
    static constexpr int kG = (GT * FP + 6 * GT + 4 * 8 * GT) * 4;   // Gamma, gate rows, reductions
    static constexpr int smem = 2 * kK + 2 * stage + kG;
};

template <int DK, int P, int PK, bool GROUP>
__global__ void __launch_bounds__(256)
delta_grads(Dims d, Parts Q, Parts K, Parts O, View G, View Beta, const __nv_bfloat16* E, const __nv_bfloat16* Y, long long eps,
            const __nv_bfloat16* S, const __nv_bfloat16* D, View dQ, View dK, View dG, View dBeta) {
    using L = GradsLayout<DK, P, PK>;
    constexpr int GT = L::GT, SV = L::SV, KP = L::KP, SP = L::SP, HP = L::HP, FP = L::FP, NT = 256;
    constexpr int WM = GT / 16, WN = 8 / WM, NBA = GT / WN / 8, DKW = DK / WN, NBK = DKW / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int mi = lane >> 3, lr = lane & 7;
    const int wm = warp % WM, wn = warp / WM;
    const int grp = blockIdx.x % d.ng;
    const int bk = blockIdx.x / d.ng, b = bk / d.hk, kh = bk % d.hk;
    const int left = min(GT, seq_len(d, b) - grp * GT);
    if (left <= 0) return;
    const long long tok = (long long)grp * GT;
    const uint32_t sb = s32(smem), kt = sb, qt = sb + L::kK, st0 = sb + 2 * L::kK;
    uint8_t* tail = smem + 2 * L::kK + 2 * L::stage;
    float* gam2 = reinterpret_cast<float*>(tail);               // Gamma [GT][FP]
    float* gl = gam2 + GT * FP;                                 // g, gamma, suffix, beta, dbeta, kappa
    float* ga = gl + GT;
    float* su = ga + GT;
    float* be = su + GT;
    float* dbe = be + GT;
    float* red = dbe + 2 * GT;                                  // [3][WN][GT] partial dots, then 8 warps' <D, W>

    auto rows = [&](uint32_t dst, int pitch, const __nv_bfloat16* src, long long ts, int width) {
        const int cpr = width / 8;
        for (int x = tid; x < GT * cpr; x += NT) {
            const int row = x / cpr, col = x % cpr;
            const bool live = row < left;
            cp16(dst + row * pitch * 2 + col * 16, src + (live ? row : 0) * ts + col * 8, live);
        }
    };
#pragma unroll
    for (int p = 0; p < PK; ++p) {
        rows(kt + p * GT * KP * 2, KP, K.p + p * K.ps + b * K.bs + kh * K.hs + tok * K.ts, K.ts, DK);
        rows(qt + p * GT * KP * 2, KP, Q.p + p * Q.ps + b * Q.bs + kh * Q.hs + tok * Q.ts, Q.ts, DK);
    }
    float tq[GROUP ? NBK : 1][4], tk[GROUP ? NBK : 1][4];
    if constexpr (GROUP) {
#pragma unroll
        for (int nb = 0; nb < NBK; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) tq[nb][q] = tk[nb][q] = 0.f;
    }
    const int ns = d.dv / SV;
    const long long state = (long long)d.dv * DK;
    const int i0 = wm * 16 + g;                                 // this lane's rows: i0, i0 + 8

    for (int rr = 0; rr < (GROUP ? d.r : 1); ++rr) {
        const int h = kh * d.r + rr;
        const long long bh = (long long)b * d.h + h;
        auto issue = [&](int sl) {
            if (sl < ns) {
                const uint32_t st = st0 + (sl & 1) * L::stage;
#pragma unroll
                for (int p = 0; p < PK; ++p)
                    rows(st + p * GT * SP * 2, SP, O.p + p * O.ps + b * O.bs + h * O.hs + tok * O.ts + sl * SV, O.ts, SV);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const long long eo = p * eps + (bh * d.N + tok) * d.dv + sl * SV;
                    rows(st + L::kO + p * GT * SP * 2, SP, E + eo, d.dv, SV);
                    rows(st + L::kO + L::kE + p * GT * SP * 2, SP, Y + eo, d.dv, SV);
                    const long long so = ((bh * d.ng + grp) * P + p) * state + (long long)sl * SV * DK;
                    for (int x = tid; x < SV * DK / 8; x += NT) {
                        const int row = x / (DK / 8), col = x % (DK / 8);
                        const uint32_t to = (p * SV * KP + row * KP + col * 8) * 2;
                        cp16(st + L::kO + 2 * L::kE + to, S + so + row * DK + col * 8, true);
                        cp16(st + L::kO + 2 * L::kE + L::kS + to, D + so + row * DK + col * 8, true);
                    }
                }
            }
            cp_commit();
        };
        issue(0);
        issue(1);
        if (tid < GT) {
            const bool live = tid < left;
            gl[tid] = live ? reinterpret_cast<const float*>(G.p)[b * G.bs + h * G.hs + (tok + tid) * G.ts] : 0.f;
            be[tid] = live ? reinterpret_cast<const float*>(Beta.p)[b * Beta.bs + h * Beta.hs + (tok + tid) * Beta.ts] : 0.f;
        }
        __syncthreads();
        if (tid < GT) {
            float a = 0.f, z = 0.f;
            for (int i = 0; i <= tid; ++i) a += gl[i];
            for (int i = GT - 1; i > tid; --i) z += gl[i];
            ga[tid] = expf(a);
            su[tid] = expf(z);
        }
        {
            constexpr int PARTS = NT / GT, RP = GT / PARTS;     // row ranges per column
            const int j = tid % GT, r0 = tid / GT * RP;
            float a = 0.f;
            for (int i = j + 1; i < r0; ++i) a += gl[i];
            for (int i = r0; i < r0 + RP; ++i) {
                if (i > j) a += gl[i];
                gam2[i * FP + j] = i >= j ? expf(a) : 0.f;
            }
        }
        float aq[NBA][4] = {}, al[NBA][4] = {};                 // dZ E^T, Y E^T
        float fq[NBK][4] = {}, f4[NBK][4] = {}, f5[NBK][4] = {};  // dZ W, E D, Y W
        float dot = 0.f;
        for (int sl = 0; sl < ns; ++sl) {
            cp_wait<1>();
            __syncthreads();
            const uint32_t ot = st0 + (sl & 1) * L::stage, et = ot + L::kO, yt = et + L::kE, wt = yt + L::kE, dt = wt + L::kS;
            const uint32_t arow = ((wm * 16 + (mi & 1) * 8 + lr) * SP + (mi >> 1) * 8) * 2;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t ao[PK][4], ae[P][4], ay[P][4];
#pragma unroll
                for (int p = 0; p < PK; ++p) ldsm4(ao[p], ot + p * GT * SP * 2 + arow + kk * 32);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    ldsm4(ae[p], et + p * GT * SP * 2 + arow + kk * 32);
                    ldsm4(ay[p], yt + p * GT * SP * 2 + arow + kk * 32);
                }
#pragma unroll
                for (int n2 = 0; n2 < NBK / 2; ++n2) {
                    const uint32_t bo = ((kk * 16 + (mi & 1) * 8 + lr) * KP + wn * DKW + n2 * 16 + (mi >> 1) * 8) * 2;
#pragma unroll
                    for (int pb = 0; pb < P; ++pb) {
                        uint32_t w[4];
                        ldsm4t(w, wt + pb * SV * KP * 2 + bo);
#pragma unroll
                        for (int pa = 0; pa < PK; ++pa)
                            if (pa + pb < P) {
                                mma16816(fq[2 * n2], ao[pa], w[0], w[1]);
                                mma16816(fq[2 * n2 + 1], ao[pa], w[2], w[3]);
                            }
#pragma unroll
                        for (int pa = 0; pa + pb < P; ++pa) {
                            mma16816(f5[2 * n2], ay[pa], w[0], w[1]);
                            mma16816(f5[2 * n2 + 1], ay[pa], w[2], w[3]);
                        }
                        ldsm4t(w, dt + pb * SV * KP * 2 + bo);
#pragma unroll
                        for (int pa = 0; pa + pb < P; ++pa) {
                            mma16816(f4[2 * n2], ae[pa], w[0], w[1]);
                            mma16816(f4[2 * n2 + 1], ae[pa], w[2], w[3]);
                        }
                    }
                }
#pragma unroll
                for (int nb = 0; nb < NBA; ++nb) {
                    const int j0 = wn * (GT / WN) + nb * 8;
                    if (j0 <= wm * 16 + 15) {
#pragma unroll
                        for (int pb = 0; pb < P; ++pb) {
                            uint32_t b0, b1;
                            asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
                                         : "=r"(b0), "=r"(b1)
                                         : "r"(et + ((pb * GT + j0 + lr) * SP + kk * 16 + (mi & 1) * 8) * 2)
                                         : "memory");
#pragma unroll
                            for (int pa = 0; pa < PK; ++pa)
                                if (pa + pb < P) mma16816(aq[nb], ao[pa], b0, b1);
#pragma unroll
                            for (int pa = 0; pa + pb < P; ++pa) mma16816(al[nb], ay[pa], b0, b1);
                        }
                    }
                }
            }
            for (int x = tid; x < SV * DK / 2; x += NT) {       // <D, W> of the slice
                const uint32_t o = (x / (DK / 2) * KP + x % (DK / 2) * 2) * 2;
                float w0 = 0.f, w1 = 0.f, d0 = 0.f, d1 = 0.f;
#pragma unroll
                for (int p = P - 1; p >= 0; --p) {
                    const uint32_t a = *reinterpret_cast<const uint32_t*>(smem + (wt - sb) + p * SV * KP * 2 + o);
                    const uint32_t z = *reinterpret_cast<const uint32_t*>(smem + (dt - sb) + p * SV * KP * 2 + o);
                    w0 += lo_f(a); w1 += hi_f(a); d0 += lo_f(z); d1 += hi_f(z);
                }
                dot = fmaf(w0, d0, fmaf(w1, d1, dot));
            }
            __syncthreads();
            issue(sl + 2);
        }
        cp_wait<0>();
        // H, F as bf16 parts in shared memory; dbeta from the diagonal of Y E^T
        uint8_t* hs = smem + 2 * L::kK;
        uint8_t* fs = hs + L::kH;
        const uint32_t ht = s32(hs), ft = s32(fs);
#pragma unroll
        for (int nb = 0; nb < NBA; ++nb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = i0 + 8 * half, j = wn * (GT / WN) + nb * 8 + 2 * t;
                float hv[2], fv[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float gm = gam2[i * FP + j + q], bj = be[j + q];
                    if (i == j + q) dbe[i] = al[nb][2 * half + q];
                    hv[q] = i >= j + q ? d.scale * gm * bj * aq[nb][2 * half + q] : 0.f;
                    fv[q] = i > j + q ? -be[i] * bj * gm * al[nb][2 * half + q] : 0.f;
                }
                uint32_t o[P];
                split2<P>(hv[0], hv[1], o);
#pragma unroll
                for (int p = 0; p < P; ++p) *reinterpret_cast<uint32_t*>(hs + ((p * GT + i) * HP + j) * 2) = o[p];
                split2<P>(fv[0], fv[1], o);
#pragma unroll
                for (int p = 0; p < P; ++p) *reinterpret_cast<uint32_t*>(fs + ((p * GT + i) * HP + j) * 2) = o[p];
            }
        dot += __shfl_xor_sync(~0u, dot, 16);
        dot += __shfl_xor_sync(~0u, dot, 8);
        dot += __shfl_xor_sync(~0u, dot, 4);
        dot += __shfl_xor_sync(~0u, dot, 2);
        dot += __shfl_xor_sync(~0u, dot, 1);
        if (lane == 0) red[3 * WN * GT + warp] = dot;
        __syncthreads();
        // dQ: scale gamma (dZ W) + H K;  second and third terms of dK: -gamma beta (Y W) + F K
        {
            const float a0 = d.scale * ga[i0], a1 = d.scale * ga[i0 + 8];
            const float c0 = -ga[i0] * be[i0], c1 = -ga[i0 + 8] * be[i0 + 8];
            const float e0 = be[i0] * su[i0], e1 = be[i0 + 8] * su[i0 + 8];
#pragma unroll
            for (int nb = 0; nb < NBK; ++nb) {
                fq[nb][0] *= a0; fq[nb][1] *= a0; fq[nb][2] *= a1; fq[nb][3] *= a1;
                f5[nb][0] *= c0; f5[nb][1] *= c0; f5[nb][2] *= c1; f5[nb][3] *= c1;
                f4[nb][0] *= e0; f4[nb][1] *= e0; f4[nb][2] *= e1; f4[nb][3] *= e1;
            }
        }
        for (int jj = 0; jj <= wm; ++jj) {
            uint32_t ah[P][4], af[P][4];
            const uint32_t ao = ((wm * 16 + (mi & 1) * 8 + lr) * HP + jj * 16 + (mi >> 1) * 8) * 2;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                ldsm4(ah[p], ht + p * GT * HP * 2 + ao);
                ldsm4(af[p], ft + p * GT * HP * 2 + ao);
            }
#pragma unroll
            for (int n2 = 0; n2 < NBK / 2; ++n2)
#pragma unroll
                for (int pb = 0; pb < PK; ++pb) {
                    uint32_t w[4];
                    ldsm4t(w, kt + ((pb * GT + jj * 16 + (mi & 1) * 8 + lr) * KP + wn * DKW + n2 * 16 + (mi >> 1) * 8) * 2);
#pragma unroll
                    for (int pa = 0; pa + pb < P; ++pa) {
                        mma16816(fq[2 * n2], ah[pa], w[0], w[1]);
                        mma16816(fq[2 * n2 + 1], ah[pa], w[2], w[3]);
                        mma16816(f5[2 * n2], af[pa], w[0], w[1]);
                        mma16816(f5[2 * n2 + 1], af[pa], w[2], w[3]);
                    }
                }
        }
        // row dots with q and k
        float rho[2] = {}, kap[2] = {}, chi[2] = {};
        auto token2 = [&](uint32_t tile, int row, int col) {    // (x[row][col], x[row][col + 1]) of a token tile
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = PK - 1; p >= 0; --p) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(smem + (tile - sb) + ((p * GT + row) * KP + col) * 2);
                v.x += lo_f(w);
                v.y += hi_f(w);
            }
            return v;
        };
#pragma unroll
        for (int nb = 0; nb < NBK; ++nb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int col = wn * DKW + nb * 8 + 2 * t;
                const float2 q = token2(qt, i0 + 8 * half, col), k = token2(kt, i0 + 8 * half, col);
                rho[half] += q.x * fq[nb][2 * half] + q.y * fq[nb][2 * half + 1] + k.x * f5[nb][2 * half] + k.y * f5[nb][2 * half + 1];
                kap[half] += k.x * f4[nb][2 * half] + k.y * f4[nb][2 * half + 1];
                f5[nb][2 * half] += f4[nb][2 * half];
                f5[nb][2 * half + 1] += f4[nb][2 * half + 1];
                f4[nb][2 * half] = f4[nb][2 * half + 1] = 0.f;
            }
        // last term of dK: H^T Q + F^T K
        for (int ii = wm; ii < WM; ++ii) {
            uint32_t ah[P][4], af[P][4];
            const uint32_t ao = ((ii * 16 + (mi >> 1) * 8 + lr) * HP + wm * 16 + (mi & 1) * 8) * 2;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                ldsm4t(ah[p], ht + p * GT * HP * 2 + ao);
                ldsm4t(af[p], ft + p * GT * HP * 2 + ao);
            }
#pragma unroll
            for (int n2 = 0; n2 < NBK / 2; ++n2)
#pragma unroll
                for (int pb = 0; pb < PK; ++pb) {
                    uint32_t w[4];
                    const uint32_t bo = ((pb * GT + ii * 16 + (mi & 1) * 8 + lr) * KP + wn * DKW + n2 * 16 + (mi >> 1) * 8) * 2;
                    ldsm4t(w, qt + bo);
#pragma unroll
                    for (int pa = 0; pa + pb < P; ++pa) {
                        mma16816(f4[2 * n2], ah[pa], w[0], w[1]);
                        mma16816(f4[2 * n2 + 1], ah[pa], w[2], w[3]);
                    }
                    ldsm4t(w, kt + bo);
#pragma unroll
                    for (int pa = 0; pa + pb < P; ++pa) {
                        mma16816(f4[2 * n2], af[pa], w[0], w[1]);
                        mma16816(f4[2 * n2 + 1], af[pa], w[2], w[3]);
                    }
                }
        }
#pragma unroll
        for (int nb = 0; nb < NBK; ++nb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float2 k = token2(kt, i0 + 8 * half, wn * DKW + nb * 8 + 2 * t);
                chi[half] += k.x * f4[nb][2 * half] + k.y * f4[nb][2 * half + 1];
                f5[nb][2 * half] += f4[nb][2 * half];
                f5[nb][2 * half + 1] += f4[nb][2 * half + 1];
            }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int o = 1; o < 4; o *= 2) {
                rho[half] += __shfl_xor_sync(~0u, rho[half], o);
                kap[half] += __shfl_xor_sync(~0u, kap[half], o);
                chi[half] += __shfl_xor_sync(~0u, chi[half], o);
            }
            if (t == 0) {
                red[wn * GT + i0 + 8 * half] = rho[half];
                red[(WN + wn) * GT + i0 + 8 * half] = kap[half];
                red[(2 * WN + wn) * GT + i0 + 8 * half] = chi[half];
            }
        }
        __syncthreads();
        if (tid < GT) {                                         // sums over the column warps, in order
            float a = 0.f, k = 0.f, x = 0.f;
            for (int w = 0; w < WN; ++w) {
                a += red[w * GT + tid];
                k += red[(WN + w) * GT + tid];
                x += red[(2 * WN + w) * GT + tid];
            }
            gl[tid] = a - x;                                    // g is no longer needed
            dbe[GT + tid] = k;
        }
        __syncthreads();
        if (tid < left) {
            float a = 0.f;
            for (int w = 0; w < 8; ++w) a += red[3 * WN * GT + w];
            a *= ga[GT - 1];
            for (int j = 0; j < tid; ++j) a += dbe[GT + j];
            for (int i = tid; i < GT; ++i) a += gl[i];
            reinterpret_cast<float*>(dG.p)[b * dG.bs + h * dG.hs + (tok + tid) * dG.ts] = a;
            reinterpret_cast<float*>(dBeta.p)[b * dBeta.bs + h * dBeta.hs + (tok + tid) * dBeta.ts] = dbe[tid];
        }
        if constexpr (GROUP) {
#pragma unroll
            for (int nb = 0; nb < NBK; ++nb)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tq[nb][q] += fq[nb][q];
                    tk[nb][q] += f5[nb][q];
                }
            __syncthreads();                                    // the stages and gate rows are written again
        }
        if (!GROUP || rr == d.r - 1) {
#pragma unroll
            for (int nb = 0; nb < NBK; ++nb)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int i = i0 + 8 * half, col = wn * DKW + nb * 8 + 2 * t;
                    if (i >= left) continue;
                    const long long qo = b * dQ.bs + kh * dQ.hs + (tok + i) * dQ.ts + col, ko = b * dK.bs + kh * dK.hs + (tok + i) * dK.ts + col;
                    const float q0 = GROUP ? tq[GROUP ? nb : 0][2 * half] : fq[nb][2 * half];
                    const float q1 = GROUP ? tq[GROUP ? nb : 0][2 * half + 1] : fq[nb][2 * half + 1];
                    const float k0 = GROUP ? tk[GROUP ? nb : 0][2 * half] : f5[nb][2 * half];
                    const float k1 = GROUP ? tk[GROUP ? nb : 0][2 * half + 1] : f5[nb][2 * half + 1];
                    if constexpr (PK == 1) {
                        *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(dQ.p) + qo) = pack2(q0, q1);
                        *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(dK.p) + ko) = pack2(k0, k1);
                    } else {
                        *reinterpret_cast<float2*>(reinterpret_cast<float*>(dQ.p) + qo) = make_float2(q0, q1);
                        *reinterpret_cast<float2*>(reinterpret_cast<float*>(dK.p) + ko) = make_float2(k0, k1);
                    }
                }
        }
    }
}

// out = the sum over images of [B][n], in image order.
static __global__ void sum_images(const float* part, float* out, int B, long long n) {
    const long long x = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (x >= n) return;
    float a = 0.f;
    for (int b = 0; b < B; ++b) a += part[b * n + x];
    out[x] = a;
}

static ttt_status run_sum_images(const float* part, float* out, int B, long long n, cudaStream_t st) {
    sum_images<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(part, out, B, n);
    return check_launch(cudaGetLastError());
}

template <int DK, int P, int PK>
static ttt_status run_reverse(const Call& c, const Parts& Q, const Parts& K, const Parts& O, const uint8_t* rec, const BackOut& out) {
    constexpr int NW = 4;
    using L = ReverseLayout<DK, P, PK, NW>;
    static_assert(L::smem <= 227 * 1024, "shared memory of a reverse CTA");
    auto* k = delta_reverse<DK, P, PK, NW>;
    ttt_status st = check_launch(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem));
    if (st != TTT_OK) return st;
    k<<<(unsigned)(c.d.B * c.d.h * (c.d.dv / L::VW)), NW * 32, L::smem, c.stream>>>(c.d, Q, K, O, rec, c.dW1, out);
    return check_launch(cudaGetLastError());
}

template <int DK, int P, int PK, bool GROUP>
static ttt_status run_grads_t(const Call& c, const Parts& Q, const Parts& K, const Parts& O, const ChainOut& fo, const BackOut& bo) {
    using L = GradsLayout<DK, P, PK>;
    static_assert(L::smem <= 227 * 1024, "shared memory of a gradient CTA");
    auto* k = delta_grads<DK, P, PK, GROUP>;
    ttt_status st = check_launch(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem));
    if (st != TTT_OK) return st;
    k<<<(unsigned)((long long)c.d.B * c.d.hk * c.d.ng), 256, L::smem, c.stream>>>(c.d, Q, K, O, c.G, c.Beta, fo.E, bo.Y, fo.e_ps,
                                                                                 fo.S, bo.D, c.dQ, c.dK, c.dG, c.dBeta);
    return check_launch(cudaGetLastError());
}
template <int DK, int P, int PK>
static ttt_status run_grads(const Call& c, const Parts& Q, const Parts& K, const Parts& O, const ChainOut& fo, const BackOut& bo) {
    return c.d.r > 1 ? run_grads_t<DK, P, PK, true>(c, Q, K, O, fo, bo) : run_grads_t<DK, P, PK, false>(c, Q, K, O, fo, bo);
}
