// delta_backward.cuh -- backward pass of the gated delta rule (included by delta.cu, inside ttt::gd).
//
// With D the adjoint of the state, y_t = D_t k_t that of the update u_t = beta_t e_t, and dz' = scale dz:
//   reverse (two warps per 16 rows of D, sequential from the last chunk to the first):
//     dU = diag(Gamma_C.) K D^T + A^T dZ,   Y = T_u^T dU  with T_u = (I + diag(beta) G)^{-1},
//     dV = diag(beta) Y,   D <- gamma_C D + (diag(gamma) dZ')^T Q - (diag(gamma) dV)^T K;
//   grads (one CTA per image, value head and group of tokens, all at once), from E, Y (per token), W at the
//     group's start and D at its end, with the group's own gamma and Gamma:
//     H_ij = scale Gamma_ij beta_j dz_i.e_j (j <= i),   F_ij = -beta_i beta_j Gamma_ij y_i.e_j (j < i),
//     dQ_i = scale gamma_i W^T dz_i + sum_j H_ij k_j,
//     dK_i = beta_i Gamma_Ci D^T e_i - gamma_i beta_i W^T y_i + sum_j F_ij k_j + sum_j (H_ji q_j + F_ji k_j),
//     dbeta_i = y_i.e_i,
//     dg_l = gamma_C <D, W> + sum_{j<l} k_j.(first term of dK_j) + sum_{i>=l} (q_i.(first term of dQ_i) + k_i.(second term of dK_i))
//            + sum_{i>=l>j} (H_ij q_i.k_j + F_ij k_i.k_j).
//   (Each term of dg_l is what one path through the gate of token l gives, so that all of them fade with the gate: sums over a token's own
//   write and readout, which a strong gate does not touch, would leave only their rounding.)
//   E and W come from the forward chain run again (they are not kept from the forward call).
// The two sequential sweeps need nothing of each other and run side by side in one launch (24 ragged heads of up to
// 1531 tokens, d = 128: 127 us).
// Every inexact operand is three bf16 parts, as in the forward pass.  (Two parts throughout were off by 3e-6 (dW0) to 6e-6 (dbeta) in the
// 2-norm, a plain fp32 computation by 1 to 3e-7.)

struct BackOut {
    View dV;
    __nv_bfloat16* Y;             // [P][B][h][N][dv]
    long long y_ps;
    __nv_bfloat16* D;             // adjoints at the groups' ends [B][h][ng][P][dv][dk]
    float* dW0;                   // nullable [B][h][dv][dk]
};

template <int DK, int PK, int RT, int KS>
struct ReverseLayout {
    static constexpr int VW = RT * 16, VB = VW * 2;
    static constexpr int kK = PK * CT * DK * 2;                // K, Q and T_u of the period's chunk,
    static constexpr int kO1 = CT * VB, kO = PK * kO1;         // dZ and A of the next one
    static constexpr int stage = (2 * kK + kO + 2 * kMat + 1023) / 1024 * 1024;
    static constexpr int kGates = kGateSlots * kGateBytes;
    static constexpr int kS = DK / 16 * P * 512;               // a tile's adjoint as operand parts
    static constexpr int kE = 2048;                            // Y, A^T dZ, partial sums
    static constexpr int kF = 2 * P * 512;                     // scale gamma dZ as operand parts
    static constexpr int kX = KS > 1 ? RT * KS * kE : 0;
    static constexpr int kOut = RT * kHelp * P * 16 * 48;
    static constexpr int fixed = kCtlBytes + kGates + 2 * RT * (kS + 2 * kE + kF) + kX + kOut + 1024;
    static constexpr int kStages = 3 * stage + fixed <= 227 * 1024 ? 3 : 2;
    static constexpr int smem = kStages * stage + fixed;
    static_assert(VB <= 128 && kK % 1024 == 0 && kO1 % 1024 == 0, "swizzled tiles");
};

// Periods k = -1 .. chunks, chunks counted from the last.  In period k the chain warps take chunk k; the helpers
// prepare what chunk k + 1 needs of dZ alone (A^T dZ, and scale gamma dZ as operand parts) and write what chunk
// k - 1 gave (Y, dV, and the adjoint it started from).
template <int DK, int PK, int RT, int KS>
__device__ __forceinline__ void reverse_body(const Dims& d, const Tiled& Q, const Tiled& K, const Tiled& O, const uint8_t* rec, const float* dW1,
                                             const BackOut& out, uint32_t* err, unsigned long long wait_ns, int block) {
    using L = ReverseLayout<DK, PK, RT, KS>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (s32(smem_raw) & 1023));
    constexpr int DW = DK / KS, KB = DW / 16, NBW = 4 / KS, CW = RT * KS, HW = RT * kHelp;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = lane & 3;
    const int slices = d.dv / L::VW;
    const int slice = block % slices;
    const int bh = block / slices, b = bh / d.h, h = bh % d.h;
    pdl_wait_primary();
    const int len = seq_len(d, b), nch = (len + CT - 1) / CT;
    const int v0 = slice * L::VW;
    const long long state = (long long)d.dv * DK;
    const uint32_t sb = s32(smem), gates = sb + L::kStages * L::stage;
    const uint32_t sbuf = gates + L::kGates, ybuf = sbuf + 2 * RT * L::kS, abuf = ybuf + 2 * RT * L::kE, fbuf = abuf + 2 * RT * L::kE,
                   xbuf = fbuf + 2 * RT * L::kF, obuf = xbuf + L::kX;
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem + L::smem - 1024 - kCtlBytes);
    auto gate_slot = [&](int k) { return gates + (k & (kGateSlots - 1)) * kGateBytes; };
    auto stage_of = [&](int k) { return sb + ((k + 1) % L::kStages) * L::stage; };

    if (warp == CW + HW) {
        // ---------------------------------------------------------------- loads
        const int recb = rec_bytes(true);
        const Abort ab{&ctl.abort_flag, err, wait_ns};
        if (lane == 0) {
            ctl.abort_flag = 0;
            for (int i = 0; i < L::kStages; ++i) mbar_init(&ctl.full[i], 1);
            fence_barrier_init();
        }
        __syncwarp();
        auto issue = [&](int k) {
            if (k >= nch) return;
            const uint32_t st = stage_of(k);
            const Loader l{&ctl.full[(k + 1) % L::kStages], lane};
            const bool now = k >= 0, next = k + 1 < nch;
            if (!now && !next) return;
            const int c = nch - 1 - k;                // the chunk of this period; the next one is c - 1
            if (lane == 0) {
                fence_proxy_async_smem();             // the warp's own stores to the stage, before the copies' writes
                uint32_t n = 0;
                if (now) n += Loader::bytes(K, len - c * CT, L::kK) + Loader::bytes(Q, len - c * CT, L::kK) + kMat;
                if (next) n += Loader::bytes(O, len - (c - 1) * CT, L::kO) + kGateBytes + kMat;
                mbar_arrive_expect_tx(l.bar, n);
            }
            __syncwarp();
            if (now) {
                load_tokens<DK, PK>(l, st, K, b, h / d.r, c * CT, len - c * CT);
                load_tokens<DK, PK>(l, st + L::kK, Q, b, h / d.r, c * CT, len - c * CT);
                l.flat(st + 2 * L::kK + L::kO, rec + ((long long)bh * d.nc + c) * recb + kGateBytes + 2 * kMat, kMat);
            }
            if (next) {
                const uint8_t* r = rec + ((long long)bh * d.nc + c - 1) * recb;
#pragma unroll
                for (int p = 0; p < PK; ++p)
                    l.template tile<L::VB, 2>(st + 2 * L::kK + p * L::kO1, O, p, b, h, (c - 1) * CT, v0, len - (c - 1) * CT);
                l.flat(gate_slot(k + 1), r, kGateBytes);
                l.flat(st + 2 * L::kK + L::kO + kMat, r + kGateBytes + kMat, kMat);
            }
        };
        for (int k = -1; k < L::kStages - 2; ++k) issue(k);
        int good = nch + 1;                           // periods before the first whose loads did not come in time
        for (int k = -1; k <= nch; ++k) {
            if (k < good && k < nch && nch > 0 && !__all_sync(~0u, mbar_wait(&ctl.full[(k + 1) % L::kStages], ((k + 1) / L::kStages) & 1, ab)))
                good = k;
            __syncthreads();
            if (k < good) issue(k + L::kStages - 1);
        }
        for (int k = good; k < nch && k < good + L::kStages - 1; ++k)        // nothing may still be on its way when the CTA ends
            mbar_drain(&ctl.full[(k + 1) % L::kStages], ((k + 1) / L::kStages) & 1, drain_limit(ab));
        return;
    }
    if (warp >= CW) {
        // ---------------------------------------------------------------- helpers
        const int hw = warp - CW, rt = hw % RT, z = hw / RT, row0 = v0 + rt * 16;
        const uint32_t stagebuf = obuf + hw * P * 16 * 48;
        for (int k = -1; k <= nch; ++k) {
            __syncthreads();
            if (k + 1 < nch) {
                const int n = k + 1, mi = lane >> 3, lr = lane & 7;
                const uint32_t st = stage_of(k), ot = st + 2 * L::kK, am = ot + L::kO + kMat, gt = gate_slot(n);
                uint32_t o[2][PK][4];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int p = 0; p < PK; ++p)
                        ldsm4t(o[kk][p], ot + p * L::kO1 + swz<L::VB>(kk * 16 + (mi >> 1) * 8 + lr, rt * 32 + (mi & 1) * 16));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float acc[4] = {};
                    mat_block<PK, false>(acc, o, am, 2 * z + i, lane);
                    sts4(abuf + ((n & 1) * RT + rt) * L::kE + ((2 * z + i) * 32 + lane) * 16, acc);
                }
                // tokens 16 z + 2t (+1), then + 8; none behind the end of the sequence
                float f[2][4];
                const int tl = len - (nch - 1 - n) * CT - z * 16 - 2 * t;
                const float2 g0 = lds2(gt + (z * 16 + 2 * t) * 4), g1 = lds2(gt + (z * 16 + 8 + 2 * t) * 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float lo = 0.f, hi = 0.f;
#pragma unroll
                    for (int p = PK - 1; p >= 0; --p) {
                        const uint32_t w = z ? o[1][p][q] : o[0][p][q];
                        lo += lo_f(w);
                        hi += hi_f(w);
                    }
                    f[q >> 1][2 * (q & 1)] = 8 * (q >> 1) < tl ? lo * (d.scale * ((q >> 1) ? g1.x : g0.x)) : 0.f;
                    f[q >> 1][2 * (q & 1) + 1] = 8 * (q >> 1) + 1 < tl ? hi * (d.scale * ((q >> 1) ? g1.y : g0.y)) : 0.f;
                }
                uint32_t a[P][4];
                as_operand(a, f[0], f[1]);
#pragma unroll
                for (int p = 0; p < P; ++p) sts4u(fbuf + ((n & 1) * RT + rt) * L::kF + ((z * P + p) * 32 + lane) * 16, a[p]);
            }
            if (k >= 1) {
                const int n = k - 1, c = nch - 1 - n, left = len - c * CT;
                const uint32_t yp = ybuf + ((n & 1) * RT + rt) * L::kE, gt = gate_slot(n);
                const float4 v = lds4(yp + (2 * z * 32 + lane) * 16), w = lds4(yp + ((2 * z + 1) * 32 + lane) * 16);
                const float y0[4] = {v.x, v.y, v.z, v.w}, y1[4] = {w.x, w.y, w.z, w.w};
                put_pair_parts(stagebuf, y0, y1, out.Y + ((long long)bh * d.N + (long long)c * CT + z * 16) * d.dv + row0, out.y_ps,
                                  d.dv, left - z * 16, lane);
                const float2 b0 = lds2(gt + (2 * CT + z * 16 + 2 * t) * 4), b1 = lds2(gt + (2 * CT + z * 16 + 8 + 2 * t) * 4);
                const float d0[4] = {b0.x * v.x, b0.y * v.y, b0.x * v.z, b0.y * v.w};
                const float d1[4] = {b1.x * w.x, b1.y * w.y, b1.x * w.z, b1.y * w.w};
                put_pair_tokens<PK>(stagebuf, d0, d1, out.dV.p,
                                    b * out.dV.bs + h * out.dV.hs + ((long long)c * CT + z * 16) * out.dV.ts + row0, out.dV.ts, left - z * 16,
                                    lane);
                if (n == 0 || ((c + 1) * CT) % d.gt == 0)
                    put_state_parts<DK>(sbuf + ((n & 1) * RT + rt) * L::kS,
                                           out.D + ((long long)bh * d.ng + (c * CT) / d.gt) * P * state, d.dv, row0, z, lane);
            }
        }
        return;
    }
    // -------------------------------------------------------------------- chain
    const int ks = warp % KS, rt = warp / KS, col0 = ks * DW, row0 = v0 + rt * 16;
    const uint32_t xp = xbuf + rt * KS * L::kE;
    float s[DW / 8][4];
    get_state<DK, DW>(s, dW1 ? dW1 + bh * state : nullptr, row0, col0, lane);
    for (int k = -1; k <= nch; ++k) {
        __syncthreads();
        if (k < 0 || k >= nch) continue;
        const int c = nch - 1 - k;
        const uint32_t st = stage_of(k), kt = st, qt = st + L::kK, um = st + 2 * L::kK + L::kO, gt = gate_slot(k);
        const uint32_t sp = sbuf + ((k & 1) * RT + rt) * L::kS, yp = ybuf + ((k & 1) * RT + rt) * L::kE,
                       ap = abuf + ((k & 1) * RT + rt) * L::kE, fp = fbuf + ((k & 1) * RT + rt) * L::kF;
        const bool hand = k == 0 || ((c + 1) * CT) % d.gt == 0;

        // dU = suffix (D K^T) + A^T dZ
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
        }
        // D <- gamma_C D + (scale gamma dZ)^T Q
        uint32_t a[2][P][4];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const uint4 v = lds4u(fp + ((kk * P + p) * 32 + lane) * 16);
                a[kk][p][0] = v.x; a[kk][p][1] = v.y; a[kk][p][2] = v.z; a[kk][p][3] = v.w;
            }
        fade_add_outer<DK, DW, PK>(s, lds1(gt + (CT - 1) * 4), a, qt, col0, lane);
        if constexpr (KS > 1) {
            tile_sync<KS>(rt);
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) sum_partials<KS>(x[nb], xp, nb, lane);
        }
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            const float2 su = lds2(gt + (CT + nb * 8 + 2 * t) * 4);
            const float4 v = lds4(ap + (nb * 32 + lane) * 16);
            x[nb][0] = fmaf(su.x, x[nb][0], v.x);
            x[nb][1] = fmaf(su.y, x[nb][1], v.y);
            x[nb][2] = fmaf(su.x, x[nb][2], v.z);
            x[nb][3] = fmaf(su.y, x[nb][3], v.w);
        }
        // Y = T_u^T dU
        float y[4][4] = {};
        as_operand(a[0], x[0], x[1]);
        as_operand(a[1], x[2], x[3]);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) mat_block<P, false>(y[nb], a, um, nb, lane);
        // D -= (gamma beta Y)^T K
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
            if (nb / NBW == ks) sts4(yp + (nb * 32 + lane) * 16, y[nb]);
            const float2 be = lds2(gt + (2 * CT + nb * 8 + 2 * t) * 4), ga = lds2(gt + (nb * 8 + 2 * t) * 4);
            const float u0 = -ga.x * be.x, u1 = -ga.y * be.y;
            y[nb][0] *= u0; y[nb][1] *= u1; y[nb][2] *= u0; y[nb][3] *= u1;
        }
        as_operand(a[0], y[0], y[1]);
        as_operand(a[1], y[2], y[3]);
        fade_add_outer<DK, DW, PK>(s, 1.f, a, kt, col0, lane);
    }
    if (out.dW0) put_state<DK, DW>(s, out.dW0 + bh * state, row0, col0, lane);
}

// The backward pass's two sequential kernels need only the prep kernel: one launch runs both, the longer one first.
struct BothArgs {
    Dims d;
    Tiled Q, K, V, O;
    const uint8_t* rec;
    const float *W0, *dW1;
    long long w0_bs;
    ChainOut chain;
    BackOut back;
    uint32_t* err;
    unsigned long long wait_ns;
    int half;                     // CTAs of each
};
template <int DK, int PK, int RT, int KS>
__global__ void __launch_bounds__(seq_warps<RT, KS>() * 32)
delta_both(const __grid_constant__ BothArgs a) {
    pdl_launch_dependents();
    if ((int)blockIdx.x < a.half)
        reverse_body<DK, PK, RT, KS>(a.d, a.Q, a.K, a.O, a.rec, a.dW1, a.back, a.err, a.wait_ns, blockIdx.x);
    else
        chain_body<DK, PK, RT, KS, true>(a.d, a.Q, a.K, a.V, a.rec, a.W0, a.w0_bs, a.chain, a.err, a.wait_ns, blockIdx.x - a.half);
}

// --------------------------------------------------------------------------------------------------
// Token gradients
// --------------------------------------------------------------------------------------------------
template <int DK, int PK>
struct GradsLayout {
    static constexpr int GT = PK == 3 ? 32 : 64;                // tokens per group
    static constexpr int SV = 32;                               // value features per slice
    static constexpr int KP = DK + 8, SP = SV + 8, HP = GT + 8, FP = GT + 1;
    static constexpr int kK = PK * GT * KP * 2;                 // K, and Q
    static constexpr int kO = PK * GT * SP * 2;
    static constexpr int kE = P * GT * SP * 2;                 // E, and Y
    static constexpr int kS = P * SV * KP * 2;                 // W, and D
    static constexpr int stage = kO + 2 * kE + 2 * kS;
    static constexpr int kH = P * GT * HP * 2;                // H, and F: in the stages' memory after the slices
    static constexpr int WM = GT / 16, WN = 8 / WM;             // warps along the tokens, and along the columns
    static constexpr int kRed = (2 * WN + WM) * GT + 8;         // partial row and column sums, then 8 warps' <D, W>
    static constexpr int kG = (GT * FP + 5 * GT) * 4;           // Gamma, gate rows and dbeta
    static_assert(2 * kH + kRed * 4 <= 2 * stage, "H, F and the sums fit the stages");
    static constexpr int smem = 2 * kK + 2 * stage + kG;
    static_assert(smem <= 227 * 1024, "shared memory of a gradient CTA");
};

// (c0, c1) += a * (b[.][0], b[.][1]), (b[.][2], b[.][3]): 16 x 16 times 16 x 16 of NA and NB parts, products of parts below the MOST-th
// dropped; summed in accumulators of their own, the small products first, and added in fp32.
template <int MOST, int NA, int NB>
__device__ __forceinline__ void add_product(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4], const uint32_t (&b)[NB][4]) {
    float u0[4] = {}, u1[4] = {};
#pragma unroll
    for (int order = MOST - 1; order >= 0; --order)
#pragma unroll
        for (int pb = 0; pb < NB; ++pb) {
            const int pa = order - pb;
            if (pa < 0 || pa >= NA) continue;
            mma16816(u0, a[pa], b[pb][0], b[pb][1]);
            mma16816(u1, a[pa], b[pb][2], b[pb][3]);
        }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        c0[q] += u0[q];
        c1[q] += u1[q];
    }
}

struct GradsArgs {
    Dims d;
    Parts Q, K, O;
    View G, Beta;
    const __nv_bfloat16 *E, *Y;       // [P][B][h][N][dv], parts eps apart
    long long eps;
    const __nv_bfloat16 *S, *D;       // states at the groups' starts, adjoints at their ends [B][h][ng][P][dv][dk]
    View dQ, dK, dG, dBeta;
    float* part;                      // nullable: fp32 dQ, then dK, per value head [2][B][h][N][dk] instead
};

// Bound: latency, one CTA of eight warps per SM (the tensor pipe is busy 38 % of the time).  32 heads of
// 4096 tokens, d = 128: 470 us.
template <int DK, int PK>
__global__ void __launch_bounds__(256)
delta_grads(const __grid_constant__ GradsArgs p) {
    using L = GradsLayout<DK, PK>;
    constexpr int GT = L::GT, SV = L::SV, KP = L::KP, SP = L::SP, HP = L::HP, FP = L::FP, NT = 256;
    constexpr int WM = L::WM, WN = L::WN, NBA = GT / WN / 8, DKW = DK / WN, NBK = DKW / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    const Dims& d = p.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int mi = lane >> 3, lr = lane & 7;
    const int wm = warp % WM, wn = warp / WM;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int grp = blockIdx.x % d.ng;
    const long long bh = blockIdx.x / d.ng;
    const int h = (int)(bh % d.h), b = (int)(bh / d.h), kh = h / d.r;
    const int left = min(GT, seq_len(d, b) - grp * GT);
    if (left <= 0) return;
    const long long tok = (long long)grp * GT;
    const uint32_t sb = s32(smem), kt = sb, qt = sb + L::kK, st0 = sb + 2 * L::kK;
    float* gam2 = reinterpret_cast<float*>(smem + 2 * L::kK + 2 * L::stage);   // Gamma [GT][FP]
    float* gl = gam2 + GT * FP;                                 // g, gamma, suffix, beta, dbeta
    float* ga = gl + GT;
    float* su = ga + GT;
    float* be = su + GT;
    float* dbe = be + GT;
    uint8_t* hs = smem + 2 * L::kK;                             // H, F, and the sums, once the slices are done
    uint8_t* fs = hs + L::kH;
    float* rows_sum = reinterpret_cast<float*>(fs + L::kH);     // [WN][GT] row terms, [WN][GT] k.(first term of dK)
    float* kap_sum = rows_sum + WN * GT;
    float* cols_sum = kap_sum + WN * GT;                        // [WM][GT] column sums
    float* dots = cols_sum + WM * GT;

    auto rows = [&](uint32_t dst, int pitch, const __nv_bfloat16* src, long long ts, int width) {
        const int cpr = width / 8;
        for (int x = tid; x < GT * cpr; x += NT) {
            const int row = x / cpr, col = x % cpr;
            const bool live = row < left;
            cp16(dst + row * pitch * 2 + col * 16, src + (live ? row : 0) * ts + col * 8, live);
        }
    };
#pragma unroll
    for (int q = 0; q < PK; ++q) {
        rows(kt + q * GT * KP * 2, KP, p.K.p + q * p.K.ps + b * p.K.bs + kh * p.K.hs + tok * p.K.ts, p.K.ts, DK);
        rows(qt + q * GT * KP * 2, KP, p.Q.p + q * p.Q.ps + b * p.Q.bs + kh * p.Q.hs + tok * p.Q.ts, p.Q.ts, DK);
    }
    const int ns = d.dv / SV;
    const long long state = (long long)d.dv * DK, so0 = (bh * d.ng + grp) * P * state;
    const int i0 = wm * 16 + g;                                 // this lane's rows: i0, i0 + 8

    auto issue = [&](int sl) {
        if (sl < ns) {
            const uint32_t st = st0 + (sl & 1) * L::stage, et = st + L::kO, yt = et + L::kE, wt = yt + L::kE, dt = wt + L::kS;
#pragma unroll
            for (int q = 0; q < PK; ++q)
                rows(st + q * GT * SP * 2, SP, p.O.p + q * p.O.ps + b * p.O.bs + h * p.O.hs + tok * p.O.ts + sl * SV, p.O.ts, SV);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const long long eo = q * p.eps + (bh * d.N + tok) * d.dv + sl * SV;
                rows(et + q * GT * SP * 2, SP, p.E + eo, d.dv, SV);
                rows(yt + q * GT * SP * 2, SP, p.Y + eo, d.dv, SV);
                const long long so = so0 + q * state + (long long)sl * SV * DK;
                for (int x = tid; x < SV * DK / 8; x += NT) {
                    const int row = x / (DK / 8), col = x % (DK / 8);
                    const uint32_t to = (q * SV * KP + row * KP + col * 8) * 2;
                    cp16(wt + to, p.S + so + row * DK + col * 8, true);
                    cp16(dt + to, p.D + so + row * DK + col * 8, true);
                }
            }
        }
        cp_commit();
    };
    issue(0);
    issue(1);
    if (tid < GT) {
        const bool live = tid < left;
        gl[tid] = live ? reinterpret_cast<const float*>(p.G.p)[b * p.G.bs + h * p.G.hs + (tok + tid) * p.G.ts] : 0.f;
        be[tid] = live ? reinterpret_cast<const float*>(p.Beta.p)[b * p.Beta.bs + h * p.Beta.hs + (tok + tid) * p.Beta.ts] : 0.f;
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
        constexpr int PARTS = NT / GT, RP = GT / PARTS;         // row ranges per column
        const int j = tid % GT, r0 = tid / GT * RP;
        float a = 0.f;
        for (int i = j + 1; i < r0; ++i) a += gl[i];
        for (int i = r0; i < r0 + RP; ++i) {
            if (i > j) a += gl[i];
            gam2[i * FP + j] = i >= j ? expf(a) : 0.f;
        }
    }
    float aq[NBA][4] = {}, al[NBA][4] = {};                     // dZ E^T, Y E^T
    float fq[NBK][4] = {}, f4[NBK][4] = {}, f5[NBK][4] = {};    // dZ W, E D, Y W
    float dot = 0.f;
    // 16 x 16 blocks (8 columns where a warp has no more) of the token by token matrices: this warp's are n = 0, 2, ..
    constexpr int NB2 = NBA > 1 ? 2 : 1;
    auto columns = [&](uint32_t (&x)[4], uint32_t tile, int pitch, int nb, int kk) {
        const int j0 = wn * (GT / WN) + nb * 8;
        if constexpr (NB2 == 2) {
            ldsm4(x, tile + ((j0 + (mi >> 1) * 8 + lr) * pitch + kk * 16 + (mi & 1) * 8) * 2);
        } else {
            asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
                         : "=r"(x[0]), "=r"(x[1])
                         : "r"(tile + ((j0 + lr) * pitch + kk * 16 + (mi & 1) * 8) * 2)
                         : "memory");
            x[2] = x[3] = 0;
        }
    };
    float none[4] = {};
    for (int sl = 0; sl < ns; ++sl) {
        cp_wait<1>();
        __syncthreads();
        const uint32_t ot = st0 + (sl & 1) * L::stage, et = ot + L::kO, yt = et + L::kE, wt = yt + L::kE, dt = wt + L::kS;
        const uint32_t arow = ((wm * 16 + (mi & 1) * 8 + lr) * SP + (mi >> 1) * 8) * 2;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t ao[PK][4], ae[P][4], ay[P][4];
#pragma unroll
            for (int q = 0; q < PK; ++q) ldsm4(ao[q], ot + q * GT * SP * 2 + arow + kk * 32);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                ldsm4(ae[q], et + q * GT * SP * 2 + arow + kk * 32);
                ldsm4(ay[q], yt + q * GT * SP * 2 + arow + kk * 32);
            }
#pragma unroll
            for (int n2 = 0; n2 < NBK / 2; ++n2) {
                const uint32_t bo = ((kk * 16 + (mi & 1) * 8 + lr) * KP + wn * DKW + n2 * 16 + (mi >> 1) * 8) * 2;
                uint32_t w[P][4];
#pragma unroll
                for (int q = 0; q < P; ++q) ldsm4t(w[q], wt + q * SV * KP * 2 + bo);
                add_product<P>(fq[2 * n2], fq[2 * n2 + 1], ao, w);
                add_product<P>(f5[2 * n2], f5[2 * n2 + 1], ay, w);
#pragma unroll
                for (int q = 0; q < P; ++q) ldsm4t(w[q], dt + q * SV * KP * 2 + bo);
                add_product<P>(f4[2 * n2], f4[2 * n2 + 1], ae, w);
            }
#pragma unroll
            for (int nb = 0; nb < NBA; nb += NB2) {
                if (wn * (GT / WN) + nb * 8 > wm * 16 + 15) continue;
                uint32_t x[P][4];
#pragma unroll
                for (int q = 0; q < P; ++q) columns(x[q], et + q * GT * SP * 2, SP, nb, kk);
                add_product<P>(aq[nb], NB2 > 1 ? aq[nb + NB2 - 1] : none, ao, x);
                add_product<P>(al[nb], NB2 > 1 ? al[nb + NB2 - 1] : none, ay, x);
            }
        }
        for (int x = tid; x < SV * DK / 2; x += NT) {           // <D, W> of the slice
            const uint32_t o = (x / (DK / 2) * KP + x % (DK / 2) * 2) * 2;
            float w0 = 0.f, w1 = 0.f, d0 = 0.f, d1 = 0.f;
#pragma unroll
            for (int q = P - 1; q >= 0; --q) {
                const uint32_t a = *reinterpret_cast<const uint32_t*>(smem + (wt - sb) + q * SV * KP * 2 + o);
                const uint32_t z = *reinterpret_cast<const uint32_t*>(smem + (dt - sb) + q * SV * KP * 2 + o);
                w0 += lo_f(a); w1 += hi_f(a); d0 += lo_f(z); d1 += hi_f(z);
            }
            dot = fmaf(w0, d0, fmaf(w1, d1, dot));
        }
        __syncthreads();
        issue(sl + 2);
    }
    cp_wait<0>();
    // H, F as bf16 parts in shared memory; dbeta from the diagonal of Y E^T; the sums of H_ij q_i.k_j + F_ij k_i.k_j along rows and columns
    const uint32_t ht = s32(hs), ft = s32(fs);
    float rho[2] = {}, kap[2] = {};
#pragma unroll
    for (int nb = 0; nb < NBA; nb += NB2) {
        float qk[2][4] = {}, kk2[2][4] = {};
        if (wn * (GT / WN) + nb * 8 <= wm * 16 + 15) {
            const uint32_t arow = ((wm * 16 + (mi & 1) * 8 + lr) * KP + (mi >> 1) * 8) * 2;
#pragma unroll(PK == 1 ? 4 : 1)
            for (int kk = 0; kk < DK / 16; ++kk) {
                uint32_t x[PK][4], a[PK][4];
#pragma unroll
                for (int q = 0; q < PK; ++q) {
                    columns(x[q], kt + q * GT * KP * 2, KP, nb, kk);
                    ldsm4(a[q], qt + q * GT * KP * 2 + arow + kk * 32);
                }
                add_product<PK>(qk[0], qk[1], a, x);
#pragma unroll
                for (int q = 0; q < PK; ++q) ldsm4(a[q], kt + q * GT * KP * 2 + arow + kk * 32);
                add_product<PK>(kk2[0], kk2[1], a, x);
            }
        }
#pragma unroll
        for (int n = 0; n < NB2; ++n) {
            const int j = wn * (GT / WN) + (nb + n) * 8 + 2 * t;
            float col[2] = {};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = i0 + 8 * half;
                float hv[2], fv[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float gm = gam2[i * FP + j + q], bj = be[j + q], y = al[nb + n][2 * half + q];
                    if (i == j + q) dbe[i] = y;
                    hv[q] = i >= j + q ? d.scale * gm * bj * aq[nb + n][2 * half + q] : 0.f;
                    fv[q] = i > j + q ? -be[i] * bj * gm * y : 0.f;
                    const float pair = i > j + q ? hv[q] * qk[n][2 * half + q] + fv[q] * kk2[n][2 * half + q] : 0.f;
                    rho[half] += pair;
                    col[q] += pair;
                }
                uint32_t o[P], f[P];
                split2(hv[0], hv[1], o);
#pragma unroll
                for (int q = 0; q < P; ++q) *reinterpret_cast<uint32_t*>(hs + ((q * GT + i) * HP + j) * 2) = o[q];
                split2(fv[0], fv[1], f);
#pragma unroll
                for (int q = 0; q < P; ++q) *reinterpret_cast<uint32_t*>(fs + ((q * GT + i) * HP + j) * 2) = f[q];
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int o = 4; o < 32; o *= 2) col[q] += __shfl_xor_sync(~0u, col[q], o);
                if (g == 0) cols_sum[wm * GT + j + q] = col[q];
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) dot += __shfl_xor_sync(~0u, dot, o);
    if (lane == 0) dots[warp] = dot;
    // First terms: scale gamma (dZ W) of dQ, beta suffix (E D) and -gamma beta (Y W) of dK, and their row dots with q and k
    auto token2 = [&](uint32_t tile, int row, int col) {        // (x[row][col], x[row][col + 1]) of a token tile
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = PK - 1; q >= 0; --q) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(smem + (tile - sb) + ((q * GT + row) * KP + col) * 2);
            v.x += lo_f(w);
            v.y += hi_f(w);
        }
        return v;
    };
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = i0 + 8 * half;
        const float fa = d.scale * ga[i], fc = -ga[i] * be[i], fe = be[i] * su[i];
#pragma unroll
        for (int nb = 0; nb < NBK; ++nb) {
            const int col = wn * DKW + nb * 8 + 2 * t;
            const float2 q = token2(qt, i, col), k = token2(kt, i, col);
            float *x = &fq[nb][2 * half], *y = &f5[nb][2 * half], *z = &f4[nb][2 * half];
            x[0] *= fa; x[1] *= fa; y[0] *= fc; y[1] *= fc; z[0] *= fe; z[1] *= fe;
            rho[half] += (q.x * x[0] + q.y * x[1]) + (k.x * y[0] + k.y * y[1]);
            kap[half] += k.x * z[0] + k.y * z[1];
            y[0] += z[0]; y[1] += z[1];
        }
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
            rho[half] += __shfl_xor_sync(~0u, rho[half], o);
            kap[half] += __shfl_xor_sync(~0u, kap[half], o);
        }
        if (t == 0) {
            rows_sum[wn * GT + i] = rho[half];
            kap_sum[wn * GT + i] = kap[half];
        }
    }
    __syncthreads();
    if (tid < GT) {                                             // sums over the warps, in order
        float a = 0.f, k = 0.f;
        for (int w = 0; w < WN; ++w) {
            a += rows_sum[w * GT + tid];
            k += kap_sum[w * GT + tid];
        }
        for (int w = 0; w < WM; ++w) a -= cols_sum[w * GT + tid];
        gl[tid] = a;                                            // g and the suffixes are no longer needed
        su[tid] = k;
    }
    for (int jj = 0; jj <= wm; ++jj) {                          // H K, F K
        uint32_t ah[P][4], af[P][4];
        const uint32_t ao = ((wm * 16 + (mi & 1) * 8 + lr) * HP + jj * 16 + (mi >> 1) * 8) * 2;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            ldsm4(ah[q], ht + q * GT * HP * 2 + ao);
            ldsm4(af[q], ft + q * GT * HP * 2 + ao);
        }
#pragma unroll
        for (int n2 = 0; n2 < NBK / 2; ++n2) {
            uint32_t w[PK][4];
#pragma unroll
            for (int q = 0; q < PK; ++q)
                ldsm4t(w[q], kt + ((q * GT + jj * 16 + (mi & 1) * 8 + lr) * KP + wn * DKW + n2 * 16 + (mi >> 1) * 8) * 2);
            add_product<P>(fq[2 * n2], fq[2 * n2 + 1], ah, w);
            add_product<P>(f5[2 * n2], f5[2 * n2 + 1], af, w);
        }
    }
    for (int ii = wm; ii < WM; ++ii) {                          // H^T Q, F^T K
        uint32_t ah[P][4], af[P][4];
        const uint32_t ao = ((ii * 16 + (mi >> 1) * 8 + lr) * HP + wm * 16 + (mi & 1) * 8) * 2;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            ldsm4t(ah[q], ht + q * GT * HP * 2 + ao);
            ldsm4t(af[q], ft + q * GT * HP * 2 + ao);
        }
#pragma unroll
        for (int n2 = 0; n2 < NBK / 2; ++n2) {
            uint32_t w[PK][4];
            const uint32_t bo = ((ii * 16 + (mi & 1) * 8 + lr) * KP + wn * DKW + n2 * 16 + (mi >> 1) * 8) * 2;
#pragma unroll
            for (int q = 0; q < PK; ++q) ldsm4t(w[q], qt + q * GT * KP * 2 + bo);
            add_product<P>(f5[2 * n2], f5[2 * n2 + 1], ah, w);
#pragma unroll
            for (int q = 0; q < PK; ++q) ldsm4t(w[q], kt + q * GT * KP * 2 + bo);
            add_product<P>(f5[2 * n2], f5[2 * n2 + 1], af, w);
        }
    }
    __syncthreads();
    if (tid < left) {
        float a = 0.f;
        for (int w = 0; w < 8; ++w) a += dots[w];
        a *= ga[GT - 1];
        for (int j = 0; j < tid; ++j) a += su[j];
        for (int i = tid; i < GT; ++i) a += gl[i];
        reinterpret_cast<float*>(p.dG.p)[b * p.dG.bs + h * p.dG.hs + (tok + tid) * p.dG.ts] = a;
        reinterpret_cast<float*>(p.dBeta.p)[b * p.dBeta.bs + h * p.dBeta.hs + (tok + tid) * p.dBeta.ts] = dbe[tid];
    }
#pragma unroll
    for (int nb = 0; nb < NBK; ++nb)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = i0 + 8 * half, col = wn * DKW + nb * 8 + 2 * t;
            if (i >= left) continue;
            const float q0 = fq[nb][2 * half], q1 = fq[nb][2 * half + 1], k0 = f5[nb][2 * half], k1 = f5[nb][2 * half + 1];
            if (p.part) {
                float* o = p.part + (bh * d.N + tok + i) * DK + col;
                *reinterpret_cast<float2*>(o) = make_float2(q0, q1);
                *reinterpret_cast<float2*>(o + (long long)d.B * d.h * d.N * DK) = make_float2(k0, k1);
                continue;
            }
            const long long qo = b * p.dQ.bs + kh * p.dQ.hs + (tok + i) * p.dQ.ts + col, ko = b * p.dK.bs + kh * p.dK.hs + (tok + i) * p.dK.ts + col;
            if constexpr (PK == 1) {
                *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.dQ.p) + qo) = pack2(q0, q1);
                *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.dK.p) + ko) = pack2(k0, k1);
            } else {
                *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.dQ.p) + qo) = make_float2(q0, q1);
                *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.dK.p) + ko) = make_float2(k0, k1);
            }
        }
}

// dQ, dK [B][hk][N][dk] (strided views; half of the grid each) = the sums over the r value heads of a key head of the fp32
// [B][h][N][dk] partial gradients, in head order.
template <bool FP32>
static __global__ void __launch_bounds__(256) sum_heads(const float* pq, const float* pk, View dQ, View dK, Dims d, long long n4) {
    pdl_wait_primary();
    const bool second = blockIdx.x >= gridDim.x / 2;
    const long long x = (blockIdx.x - (second ? gridDim.x / 2 : 0)) * 256LL + threadIdx.x;
    if (x >= n4) return;
    const float* part = second ? pk : pq;
    const View& out = second ? dK : dQ;
    const int w4 = d.dk / 4, c = (int)(x % w4) * 4;
    const long long row = x / w4;
    const int t = (int)(row % d.N), kh = (int)(row / d.N % d.hk), b = (int)(row / d.N / d.hk);
    if (t >= seq_len(d, b)) return;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < d.r; ++r) {
        const float4 v = *reinterpret_cast<const float4*>(part + (((long long)b * d.h + kh * d.r + r) * d.N + t) * d.dk + c);
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
    const long long o = b * out.bs + kh * out.hs + t * out.ts + c;
    if (FP32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(out.p) + o) = a;
    else *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(out.p) + o) = make_uint2(pack2(a.x, a.y), pack2(a.z, a.w));
}

// out = the sum over images of [B][n], in image order.
static __global__ void sum_images(const float* part, float* out, int B, long long n) {
    pdl_wait_primary();
    const long long x = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (x >= n) return;
    float a = 0.f;
    for (int b = 0; b < B; ++b) a += part[b * n + x];
    out[x] = a;
}

static ttt_status run_sum_images(const float* part, float* out, int B, long long n, cudaStream_t st) {
    return launch(sum_images, (n + 255) / 256, 256, 0, st, part, out, B, n);
}

template <int DK, int PK, int RT, int KS>
static ttt_status run_both_t(const Call& c, const Parts& Q, const Parts& K, const Parts& O, const uint8_t* rec, const ChainOut& out,
                             const BackOut& bo) {
    using R = ReverseLayout<DK, PK, RT, KS>;
    using F = ChainLayout<DK, PK, RT, KS, true>;
    constexpr int smem = R::smem > F::smem ? R::smem : F::smem;
    static_assert(smem <= 227 * 1024, "shared memory of a sequential CTA");
    constexpr auto k = delta_both<DK, PK, RT, KS>;
    const ttt_status st = allow_smem<k>(std::max(smem, kAloneSmem));
    if (st != TTT_OK) return st;
    const int half = c.d.B * c.d.h * (c.d.dv / (RT * 16));
    const BothArgs a{c.d, tiled(Q, PK, c.d, c.d.hk, DK, 128), tiled(K, PK, c.d, c.d.hk, DK, 128),
                     tiled(c.V.p, 0, 1, c.V.bs, c.V.hs, c.V.ts, c.d, c.d.h, c.d.dv, PK == 1 ? 2 : 4, F::VB),
                     tiled(O, PK, c.d, c.d.h, c.d.dv, R::VB), rec, c.W0, c.dW1, c.w0_bs, out, bo, error_word(c), c.wait_ns, half};
    return launch(k, 2LL * half, seq_warps<RT, KS>() * 32, spread_smem(smem, 2LL * half, c.sms), c.stream, a);
}
template <int DK, int PK>
static ttt_status run_both(const Call& c, const Parts& Q, const Parts& K, const Parts& O, const uint8_t* rec, const ChainOut& out,
                           const BackOut& bo) {
    // fp32: the three parts of a second tile do not fit the shared memory
    if (PK == 3 || few_tiles(c, 2)) return run_both_t<DK, PK, 1, 2>(c, Q, K, O, rec, out, bo);
    return run_both_t<DK, PK, PK == 1 ? 2 : 1, 2>(c, Q, K, O, rec, out, bo);
}

// part: fp32 workspace of the gradients per value head, used where value heads share key heads.
template <int DK, int PK>
static ttt_status run_grads(const Call& c, const Parts& Q, const Parts& K, const Parts& O, const ChainOut& fo, const BackOut& bo, float* part) {
    using L = GradsLayout<DK, PK>;
    const Dims& d = c.d;
    constexpr auto k = delta_grads<DK, PK>;
    ttt_status st = allow_smem<k>(L::smem);
    if (st != TTT_OK) return st;
    const GradsArgs a{d, Q, K, O, c.G, c.Beta, fo.E, bo.Y, fo.e_ps, fo.S, bo.D, c.dQ, c.dK, c.dG, c.dBeta, d.r > 1 ? part : nullptr};
    st = launch(k, (long long)d.B * d.h * d.ng, 256, L::smem, c.stream, a);
    if (st != TTT_OK || d.r == 1) return st;
    const long long n4 = (long long)d.B * d.hk * d.N * DK / 4, rows = (long long)d.B * d.h * d.N;
    return launch(sum_heads<PK == 3>, 2 * ((n4 + 255) / 256), 256, 0, c.stream, part, part + rows * DK, c.dQ, c.dK, d, n4);
}
