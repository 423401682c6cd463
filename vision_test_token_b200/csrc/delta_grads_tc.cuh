// delta_grads_tc.cuh -- token gradients of the gated delta rule for bf16 tokens, on tcgen05 (included by delta.cu,
// inside ttt::gd; the formulas are in delta_backward.cuh).
//
// One work item is a group of 64 tokens of one value head; CTAs (one per SM) loop over items.  Per item:
//   slices of 32 value features (TMA, two stages):
//     [dA ; dL] += [dZ ; Y] E^T         tensor memory: token rows 0-63 and 64-127, 64 columns
//     [Q1 ; K5] += [dZ ; Y] W           W: the state at the group's start, d_k columns
//     [ 0 ; K4] += [ 0 ; E] D           D: the adjoint at the group's end
//   eight elementwise warps: H and F (bf16 parts, shared memory) from dA, dL; Q1 and K5 scaled by row
//     [Q1 ; K5] += [H ; F] K,    [0 ; C] = [0 ; H^T] Q + [0 ; F^T] K
//   the same warps: dQ = Q1, dK = K5 + beta Gamma_C K4 + C, and the row dots that give dg.
// Two operands that meet the same right-hand side are stacked into one product of 128 rows (a product of 64 rows
// takes the tensor core as long); blocks of zeros keep K4 and C in the lanes of K5, so that a thread finds all
// terms of its token in its own lane.  Y, E, W, D, H and F come as two bf16 parts; the product of the two low
// parts is dropped.
//
// Bound: the latency of an item's dependent steps (one CTA per SM; about 90 products of 128 x 64-128 x 16 and 240 KB of
// operands per item).  32 heads of 4096 tokens, d = 128: 140 us, 505 MB read, HBM 49 % and the tensor pipe 34 % busy.

template <int DK>
struct GradsTc {
    static constexpr int GT = 64, SV = 32;
    static constexpr int kTok = DK / 64 * GT * 128;            // K, and Q: [half][64 tokens][128 bytes]
    static constexpr int kV = GT * 64;                         // 64 tokens x 32 features: rows of 64 bytes
    static constexpr int kSt = DK / 64 * SV * 128;             // 32 features x d_k of one part: [half][32][128 bytes]
    // a stage: dZ, Y hi | 0, Y lo | 0, E hi | 0, E lo | W hi, W lo, D hi, D lo
    static constexpr int oO = 0, oYh = kV, oZ0 = 2 * kV, oYl = 3 * kV, oZ1 = 4 * kV, oEh = 5 * kV, oZ2 = 6 * kV, oEl = 7 * kV, oW = 8 * kV,
                         oD = oW + 2 * kSt, stage = oD + 2 * kSt;
    static constexpr int loaded = 5 * kV + 4 * kSt;            // bytes that arrive per slice
    static constexpr int kH = GT * 128;                        // one part of H or F: [64][128 bytes]
    static constexpr int oK = 2 * stage, oQ = oK + kTok, oZero = oQ + kTok, oH = oZero + kH;   // H hi, F hi, H lo, F lo
    static constexpr int oMisc = oH + 4 * kH;
    static constexpr int kRow = 6 * GT + 16;                   // floats of one item's gate rows and sums
    static constexpr int kMisc = (GT * (GT + 1) + 2 * kRow + 2 * 3 * GT) * 4 + 256;
    static constexpr int smem = oMisc + kMisc + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of a gradient CTA");
    static constexpr uint32_t cA = 0, cQ = 64, cK4 = 64 + DK, cC = 64 + 2 * DK;                // tensor-memory columns
};

struct GradsArgs {
    Dims d;
    CUtensorMap K, Q, O, E, Y, S, D;      // bf16; E, Y, S, D: rows of a plain matrix
    View G, Beta, dQ, dK, dG, dBeta;
    int kh, kb, oh, ob;                   // 0 where K and Q (kh, kb; qh, qb) or dZ are broadcast over heads or images
    int qh, qb;
    int out_fp32, out_per_head;           // dQ and dK are fp32 partial sums per value head
    uint32_t* err;
    unsigned long long wait_ns;
    long long items;
};

struct GradsCtl {
    uint64_t kq_full, kq_empty, full[2], empty[2], acc_a, acc, hf, fin, rows, side[2];
    uint32_t tmem;
    int abort_flag;
};

// Shared-memory descriptor of a 64-byte-swizzled K-major operand (bf16, 32 columns): groups of 8 rows 512 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(512 >> 4) << 32) | (1ull << 46) |
           (4ull << 61);
}
template <int DK>
__global__ void __launch_bounds__(384, 1)
delta_grads_tc(const __grid_constant__ GradsArgs p) {
    using L = GradsTc<DK>;
    constexpr int GT = L::GT, SV = L::SV;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (s32(smem_raw) & 1023));
    const uint32_t sb = s32(smem);
    const Dims& d = p.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* gam2 = reinterpret_cast<float*>(smem + L::oMisc);      // Gamma [64][65]
    // rows of one item: gamma, suffix, beta, dbeta; g, its sum behind a token inside a block of 16; <D, W> per
    // side warp, the blocks' sums of g.  Two items' worth.
    float* rows = gam2 + GT * (GT + 1);
    float* red = rows + 2 * L::kRow;                              // [2 halves][3][64]
    GradsCtl& ctl = *reinterpret_cast<GradsCtl*>(red + 2 * 3 * GT);
    const Abort ab{&ctl.abort_flag, p.err, p.wait_ns};
    const int ns = d.dv / SV;

    for (int x = tid; x < L::kH / 16; x += 384) *reinterpret_cast<uint4*>(smem + L::oZero + x * 16) = make_uint4(0, 0, 0, 0);
    for (int s = 0; s < 2; ++s)
        for (int o : {L::oZ0, L::oZ1, L::oZ2})
            for (int x = tid; x < L::kV / 16; x += 384)
                *reinterpret_cast<uint4*>(smem + s * L::stage + o + x * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (tid == 0) {
        ctl.abort_flag = 0;
        mbar_init(&ctl.kq_full, 1);
        mbar_init(&ctl.kq_empty, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 3);
        }
        mbar_init(&ctl.acc_a, 1);
        mbar_init(&ctl.acc, 1);
        mbar_init(&ctl.hf, 8);
        mbar_init(&ctl.fin, 1);
        mbar_init(&ctl.rows, 2);
        // a side warp may finish the next item before an elementwise warp looks for this one: one barrier per parity (two
        // items ahead it waits for that warp's H and F)
        mbar_init(&ctl.side[0], 2);
        mbar_init(&ctl.side[1], 2);
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&ctl.tmem, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait_primary();
    __syncthreads();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;                   // all 512 columns are this CTA's: they start at 0

    // items of this CTA: group fastest, then value head, then image
    auto next_item = [&](long long& it) {          // skips groups behind the end of their sequence
        for (; it < p.items; it += gridDim.x) {
            const int grp = (int)(it % d.ng), b = (int)(it / d.ng / d.h);
            if (grp * GT < seq_len(d, b)) return true;
        }
        return false;
    };

    if (warp == 8) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            uint32_t n = 0, sl = 0, kq = 0;        // items, slices and K, Q tiles so far
            bool ok = true;
            for (long long it = blockIdx.x; ok && next_item(it); it += gridDim.x, ++n) {
                const int grp = (int)(it % d.ng);
                const long long bh = it / d.ng;
                const int h = (int)(bh % d.h), b = (int)(bh / d.h), kh = h / d.r, tok = grp * GT;
                for (int s = 0; s < ns; ++s, ++sl) {
                    if (s == 2 || ns == 2 && s == 1) {
                        // K and Q after the first slices, which do not have to wait for the last item's tail
                        if (n > 0) ok = mbar_wait(&ctl.kq_empty, (n - 1) & 1, ab);
                        if (!ok) break;
                        fence_proxy_async_smem();
                        mbar_arrive_expect_tx(&ctl.kq_full, 2 * L::kTok);
                        ++kq;
                        for (int c = 0; c < DK / 64; ++c) {
                            tma_load_5d_at(sb + L::oK + c * GT * 128, &p.K, &ctl.kq_full, c * 64, tok, kh * p.kh, b * p.kb, 0);
                            tma_load_5d_at(sb + L::oQ + c * GT * 128, &p.Q, &ctl.kq_full, c * 64, tok, kh * p.qh, b * p.qb, 0);
                        }
                    }
                    if (sl >= 2) ok = mbar_wait(&ctl.empty[sl & 1], ((sl >> 1) - 1) & 1, ab);
                    if (!ok) break;
                    uint64_t* bar = &ctl.full[sl & 1];
                    const uint32_t st = sb + (sl & 1) * L::stage;
                    mbar_arrive_expect_tx(bar, L::loaded);
                    tma_load_5d_at(st + L::oO, &p.O, bar, s * SV, tok, h * p.oh, b * p.ob, 0);
                    // rows of a part past its tensor's end belong to the next sequence or part: finite or not, they
                    // reach only rows and columns that are not used
                    const int row = (int)(bh * d.N + tok);
                    tma_load_5d_at(st + L::oYh, &p.Y, bar, s * SV, row, 0, 0, 0);
                    tma_load_5d_at(st + L::oYl, &p.Y, bar, s * SV, row, 1, 0, 0);
                    tma_load_5d_at(st + L::oEh, &p.E, bar, s * SV, row, 0, 0, 0);
                    tma_load_5d_at(st + L::oEl, &p.E, bar, s * SV, row, 1, 0, 0);
                    for (int part = 0; part < 2; ++part) {
                        const long long r = ((bh * d.ng + grp) * 2 + part) * d.dv + s * SV;
                        for (int c = 0; c < DK / 64; ++c) {
                            tma_load_5d_at(st + L::oW + part * L::kSt + c * SV * 128, &p.S, bar, c * 64, (int)r, 0, 0, 0);
                            tma_load_5d_at(st + L::oD + part * L::kSt + c * SV * 128, &p.D, bar, c * 64, (int)r, 0, 0, 0);
                        }
                    }
                }
            }
            // nothing may still be on its way when the CTA ends
            if (kq > 0) mbar_drain(&ctl.kq_full, (kq - 1) & 1, drain_limit(ab));
            for (uint32_t k = sl > 2 ? sl - 2 : 0; k < sl; ++k) mbar_drain(&ctl.full[k & 1], (k >> 1) & 1, drain_limit(ab));
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t idA = idesc_bf16_f32(128, 64, false, false);      // [.] E^T: both K-major
        constexpr uint32_t idS = idesc_bf16_f32(128, DK, false, true);       // [.] W, D, K: right side feature-major
        constexpr uint32_t idT = idesc_bf16_f32(128, DK, true, true);        // [0 ; H^T] Q
        uint32_t n = 0, sl = 0;
        bool ok = true;
        for (long long it = blockIdx.x; ok && next_item(it); it += gridDim.x, ++n) {
            if (n > 0) ok = mbar_wait(&ctl.kq_empty, (n - 1) & 1, ab);       // the accumulators have been read
            for (int s = 0; ok && s < ns; ++s, ++sl) {
                ok = mbar_wait(&ctl.full[sl & 1], (sl >> 1) & 1, ab);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t st = sb + (sl & 1) * L::stage;
                    const uint64_t aOY = sdesc_sw64(st + L::oO), aYl = sdesc_sw64(st + L::oZ0), bEh = sdesc_sw64(st + L::oEh),
                                   bEl = sdesc_sw64(st + L::oEl), aEh = sdesc_sw64(st + L::oZ1), aEl = sdesc_sw64(st + L::oZ2);
                    const uint64_t bWh = sdesc_sw128(st + L::oW, SV * 128, 1024), bWl = sdesc_sw128(st + L::oW + L::kSt, SV * 128, 1024),
                                   bDh = sdesc_sw128(st + L::oD, SV * 128, 1024), bDl = sdesc_sw128(st + L::oD + L::kSt, SV * 128, 1024);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {           // 16 features: 32 bytes of a K-major row, 16 rows of W and D
                        const uint32_t acc = s > 0 || kk > 0;
                        mma_bf16_ss(tmem + L::cA, aOY + 2 * kk, bEh + 2 * kk, idA, acc);
                        mma_bf16_ss(tmem + L::cA, aOY + 2 * kk, bEl + 2 * kk, idA, 1);
                        mma_bf16_ss(tmem + L::cA, aYl + 2 * kk, bEh + 2 * kk, idA, 1);
                    }
                    if (s == ns - 1) mma_commit(&ctl.acc_a);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const uint32_t acc = s > 0 || kk > 0;
                        mma_bf16_ss(tmem + L::cQ, aOY + 2 * kk, bWh + 128 * kk, idS, acc);
                        mma_bf16_ss(tmem + L::cQ, aOY + 2 * kk, bWl + 128 * kk, idS, 1);
                        mma_bf16_ss(tmem + L::cQ, aYl + 2 * kk, bWh + 128 * kk, idS, 1);
                        mma_bf16_ss(tmem + L::cK4, aEh + 2 * kk, bDh + 128 * kk, idS, acc);
                        mma_bf16_ss(tmem + L::cK4, aEh + 2 * kk, bDl + 128 * kk, idS, 1);
                        mma_bf16_ss(tmem + L::cK4, aEl + 2 * kk, bDh + 128 * kk, idS, 1);
                    }
                    mma_commit(&ctl.empty[sl & 1]);
                    if (s == ns - 1) mma_commit(&ctl.acc);
                }
                __syncwarp();
            }
            if (!ok) break;
            ok = mbar_wait(&ctl.hf, n & 1, ab) && mbar_wait(&ctl.kq_full, n & 1, ab);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < GT / 16; ++kk)
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint32_t hp = sb + L::oH + part * 2 * L::kH;       // H, then F
                        const uint64_t bK = sdesc_sw128(sb + L::oK + kk * 2048, GT * 128, 1024),
                                       bQ = sdesc_sw128(sb + L::oQ + kk * 2048, GT * 128, 1024);
                        mma_bf16_ss(tmem + L::cQ, sdesc_sw128(hp + kk * 32, 16, 1024), bK, idS, 1);
                        // rows 0-63 of the left side: the zero block; rows 64-127: H or F read by columns
                        const uint32_t z = sb + L::oZero + kk * 2048;
                        mma_bf16_ss(tmem + L::cC, sdesc_sw128(z, hp - (sb + L::oZero), 1024), bQ, idT, kk > 0 || part > 0);
                        mma_bf16_ss(tmem + L::cC, sdesc_sw128(z, hp + L::kH - (sb + L::oZero), 1024), bK, idT, 1);
                    }
                mma_commit(&ctl.fin);
            }
            __syncwarp();
        }
        // the last products end before the CTA gives its tensor memory back
        if (!ok) {
            if (elect_one()) mma_commit(&ctl.fin);
            __syncwarp();
            mbar_drain(&ctl.fin, n & 1, drain_limit(ab));
        } else if (n > 0) {
            mbar_drain(&ctl.fin, (n - 1) & 1, drain_limit(ab));
        }
    } else if (warp >= 10) {
        // ---------------------------------------------------------------- gates, Gamma and <D, W>
        const int sw = warp - 10, t = sw * 32 + lane;              // token (and column of Gamma) of this thread
        uint32_t n = 0, sl = 0;
        bool ok = true;
        for (long long it = blockIdx.x; ok && next_item(it); it += gridDim.x, ++n) {
            const int grp = (int)(it % d.ng);
            const long long bh = it / d.ng;
            const int h = (int)(bh % d.h), b = (int)(bh / d.h);
            const int left = min(GT, seq_len(d, b) - grp * GT);
            const long long tok = (long long)grp * GT + t;
            float *ga = rows + (n & 1) * L::kRow, *su = ga + GT, *be = su + GT, *gl = be + 2 * GT, *suf16 = gl + GT, *dots = suf16 + GT;
            const bool live = t < left;
            const float g = live ? reinterpret_cast<const float*>(p.G.p)[b * p.G.bs + h * p.G.hs + tok * p.G.ts] : 0.f;
            const float beta = live ? reinterpret_cast<const float*>(p.Beta.p)[b * p.Beta.bs + h * p.Beta.hs + tok * p.Beta.ts] : 0.f;
            auto gates_and_gamma = [&] {
                float pre = g, suf = __shfl_down_sync(~0u, g, 1);
                if (lane == 31) suf = 0.f;
                float s16 = lane % 16 == 15 ? 0.f : suf;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const float x = __shfl_up_sync(~0u, pre, o), z = __shfl_down_sync(~0u, suf, o), y = __shfl_down_sync(~0u, s16, o);
                    if (lane >= o) pre += x;
                    if (lane + o < 32) suf += z;
                    if (lane % 16 + o < 16) s16 += y;
                }
                // Gamma of the last item and the rows of the one before have been read by every warp
                if (n > 0) ok = ok && mbar_wait(&ctl.hf, (n - 1) & 1, ab);
                be[t] = beta;
                gl[t] = g;
                suf16[t] = s16;
                if (lane % 16 == 0) dots[2 + t / 16] = g + s16;
                named_bar_sync(2, 64);
                const float other = sw ? dots[2] + dots[3] : dots[4] + dots[5];      // the other half's sum of g
                ga[t] = expf(sw ? other + pre : pre);
                su[t] = expf(sw ? suf : suf + other);
                // Gamma, column t: logs summed from zero at row t
                float a = 0.f;
                for (int rb = 0; rb < 4; ++rb) {
                    if (rb == t / 16 + 1) a = s16;
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        const float4 v = *reinterpret_cast<const float4*>(gl + rb * 16 + k4 * 4);
                        const float g4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = rb * 16 + k4 * 4 + e;
                            if (k > t) a += g4[e];
                            gam2[k * (GT + 1) + t] = k >= t ? __expf(a) : 0.f;       // relative error about 2^-22 (1 + |a|)
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.rows);
            };
            float dot[2] = {0.f, 0.f};
            for (int s = 0; s < ns; ++s, ++sl) {
                if (s == 2) gates_and_gamma();     // the first two slices may be here before the last item is done
                ok = ok && mbar_wait(&ctl.full[sl & 1], (sl >> 1) & 1, ab);
                const uint8_t* st = smem + (sl & 1) * L::stage;
#pragma unroll 2
                for (int x = t; x < L::kSt / 16; x += 64) {
                    const uint4 wh = *reinterpret_cast<const uint4*>(st + L::oW + x * 16), wl = *reinterpret_cast<const uint4*>(st + L::oW + L::kSt + x * 16);
                    const uint4 dh = *reinterpret_cast<const uint4*>(st + L::oD + x * 16), dl = *reinterpret_cast<const uint4*>(st + L::oD + L::kSt + x * 16);
                    const uint32_t w0[4] = {wh.x, wh.y, wh.z, wh.w}, w1[4] = {wl.x, wl.y, wl.z, wl.w}, d0[4] = {dh.x, dh.y, dh.z, dh.w},
                                   d1[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        dot[0] = fmaf(lo_f(w0[k]) + lo_f(w1[k]), lo_f(d0[k]) + lo_f(d1[k]), dot[0]);
                        dot[1] = fmaf(hi_f(w0[k]) + hi_f(w1[k]), hi_f(d0[k]) + hi_f(d1[k]), dot[1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.empty[sl & 1]);
            }
            if (ns == 2) gates_and_gamma();
            dot[0] += dot[1];
#pragma unroll
            for (int o = 16; o > 0; o /= 2) dot[0] += __shfl_xor_sync(~0u, dot[0], o);
            if (lane == 0) {
                dots[sw] = dot[0];
                mbar_arrive(&ctl.side[n & 1]);
            }
            ok = __all_sync(~0u, ok);
        }
    } else {
        // ---------------------------------------------------------------- elementwise
        const int q = warp & 3, ch = warp >> 2;    // tensor-memory lane quarter, column half
        const uint32_t lofs = (uint32_t)(q * 32) << 16;
        const bool upper = q < 2;                  // rows of dA, Q1 (else of dL, K5, K4, C)
        const int i = (q & 1) * 32 + lane;         // token of the group
        uint32_t n = 0;
        bool ok = true;
        for (long long it = blockIdx.x; ok && next_item(it); it += gridDim.x, ++n) {
            const int grp = (int)(it % d.ng);
            const long long bh = it / d.ng;
            const int h = (int)(bh % d.h), b = (int)(bh / d.h);
            const int left = min(GT, seq_len(d, b) - grp * GT);
            const long long tok = (long long)grp * GT;
            float *ga = rows + (n & 1) * L::kRow, *su = ga + GT, *be = su + GT, *dbe = be + GT, *dots = dbe + 3 * GT;
            ok = ok && mbar_wait(&ctl.kq_full, n & 1, ab);
            // tokens behind the end of the sequence: their rows of K and Q are not the caller's, and 0 x NaN is NaN
            if (ok && left < GT) {
                for (int x = tid; x < (GT - left) * 16 * (DK / 64); x += 256) {
                    const int c = x / ((GT - left) * 16), y = x % ((GT - left) * 16);
                    const int o = c * GT * 128 + left * 128 + (y / 2) * 16;
                    *reinterpret_cast<uint4*>(smem + (y & 1 ? L::oQ : L::oK) + o) = make_uint4(0, 0, 0, 0);
                }
            }
            named_bar_sync(1, 256);
            ok = ok && mbar_wait(&ctl.rows, n & 1, ab) && mbar_wait(&ctl.acc_a, n & 1, ab);
            if (named_bar_or(1, 256, !ok)) break;
            tc_fence_after();
            {
                // H (upper) or F, columns 32 ch .. 32 ch + 31 of row i
                float v[32];
                tmem_ld<32>(tmem + L::cA + lofs + ch * 32, v);
                const float ri = i >= left ? 0.f : upper ? d.scale : -be[i];
                const int last = i >= left ? -1 : upper ? i : i - 1;   // last column of the row
                if (!upper && i / 32 == ch) {
                    float x = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) x = k == lane ? v[k] : x;
                    dbe[i] = x;
                }
#pragma unroll
                for (int j8 = 0; j8 < 4; ++j8) {
                    uint32_t hi[4], lo[4];
                    const float4 b0 = *reinterpret_cast<const float4*>(be + ch * 32 + j8 * 8),
                                 b1 = *reinterpret_cast<const float4*>(be + ch * 32 + j8 * 8 + 4);
                    const float bj[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
                    for (int j2 = 0; j2 < 4; ++j2) {
                        float w[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int jl = j8 * 8 + j2 * 2 + k, j = ch * 32 + jl;
                            w[k] = j <= last ? ri * bj[j2 * 2 + k] * gam2[i * (GT + 1) + j] * v[jl] : 0.f;
                        }
                        uint32_t o[2];
                        split2<2>(w[0], w[1], o);
                        hi[j2] = o[0];
                        lo[j2] = o[1];
                    }
                    const uint32_t o = L::oH + (upper ? 0 : L::kH) + i * 128 + (((ch * 4 + j8) ^ (i & 7)) << 4);
                    *reinterpret_cast<uint4*>(smem + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(smem + o + 2 * L::kH) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            ok = mbar_wait(&ctl.acc, n & 1, ab);
            tc_fence_after();
            {
                // Q1 by scale gamma, K5 by -gamma beta
                const float f = upper ? d.scale * ga[i] : -ga[i] * be[i];
#pragma unroll
                for (int c = 0; c < DK / 2; c += 32) {
                    const uint32_t col = tmem + L::cQ + lofs + ch * (DK / 2) + c;
                    float v[32];
                    tmem_ld<32>(col, v);
                    uint32_t w[2][16];
#pragma unroll
                    for (int k = 0; k < 32; ++k) w[k / 16][k % 16] = __float_as_uint(f * v[k]);
                    tmem_st16(col, w[0]);
                    tmem_st16(col + 16, w[1]);
                }
                tmem_st_wait();
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.hf);
            ok = ok && mbar_wait(&ctl.fin, n & 1, ab);
            if (named_bar_or(1, 256, !ok)) break;
            tc_fence_after();
            // dQ (upper) or dK, columns ch DK / 2 .. of row i, and the row dots
            float v[DK / 64][32];
            {
                float rho = 0.f, kp = 0.f, chi = 0.f;
                const float f4 = be[i] * su[i];
#pragma unroll
                for (int c = 0; c < DK / 64; ++c) {
                    const int col = ch * (DK / 2) + c * 32;
                    tmem_ld<32>(tmem + L::cQ + lofs + col, v[c]);
                    uint4 x[4];                    // the token's q or k
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int piece = col / 8 + k;
                        x[k] = *reinterpret_cast<const uint4*>(smem + (upper ? L::oQ : L::oK) + (piece >> 3) * GT * 128 + i * 128 +
                                                               (((piece & 7) ^ (i & 7)) << 4));
                    }
                    auto dotx = [&](const float (&u)[32]) {
                        float a[2] = {0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                a[0] = fmaf(lo_f(w[e]), u[k * 8 + 2 * e], a[0]);
                                a[1] = fmaf(hi_f(w[e]), u[k * 8 + 2 * e + 1], a[1]);
                            }
                        }
                        return a[0] + a[1];
                    };
                    rho += dotx(v[c]);
                    if (!upper) {
                        float u[32];
                        tmem_ld<32>(tmem + L::cK4 + lofs + col, u);
                        kp += f4 * dotx(u);
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[c][k] = fmaf(f4, u[k], v[c][k]);
                        tmem_ld<32>(tmem + L::cC + lofs + col, u);
                        chi += dotx(u);
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[c][k] += u[k];
                    }
                }
                tc_fence_before();
                if (upper) red[ch * 3 * GT + i] = rho;
                else {
                    red[ch * 3 * GT + GT + i] = rho - chi;
                    red[ch * 3 * GT + 2 * GT + i] = kp;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.kq_empty);      // K, Q and the accumulators are free
            {
                // the warp's 32 rows through its share of H and F (read by now), then whole sectors per row
                const View& ov = upper ? p.dQ : p.dK;
                const int i0 = (q & 1) * 32;       // the warp's first token
                const long long off = b * ov.bs + (p.out_per_head ? h : h / d.r) * ov.hs + (tok + i0) * ov.ts;
                const uint32_t own = L::oH + warp * 4096;
#pragma unroll
                for (int c = 0; c < DK / 64; ++c) {
                    const int col = ch * (DK / 2) + c * 32;
                    if (p.out_fp32) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4*>(smem + own + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                                make_float4(v[c][4 * k], v[c][4 * k + 1], v[c][4 * k + 2], v[c][4 * k + 3]);
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = k * 4 + lane / 8, pc = lane & 7;
                            const float4 x4 = *reinterpret_cast<const float4*>(smem + own + r * 128 + ((pc ^ (r & 7)) << 4));
                            if (i0 + r < left) *reinterpret_cast<float4*>(reinterpret_cast<float*>(ov.p) + off + r * ov.ts + col + pc * 4) = x4;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4*>(smem + own + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
                                make_uint4(pack2(v[c][8 * k], v[c][8 * k + 1]), pack2(v[c][8 * k + 2], v[c][8 * k + 3]),
                                           pack2(v[c][8 * k + 4], v[c][8 * k + 5]), pack2(v[c][8 * k + 6], v[c][8 * k + 7]));
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = k * 8 + lane / 4, pc = lane & 3;
                            const uint4 x4 = *reinterpret_cast<const uint4*>(smem + own + r * 64 + ((pc ^ ((r >> 1) & 3)) << 4));
                            if (i0 + r < left) *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(ov.p) + off + r * ov.ts + col + pc * 8) = x4;
                        }
                    }
                    __syncwarp();
                }
            }
            ok = mbar_wait(&ctl.side[n & 1], (n >> 1) & 1, ab);
            if (named_bar_or(1, 256, !ok)) break;
            if (warp == 0) {                                // dg and dbeta; the other warps go on
                float v[2], k[2], kin[2], total;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    v[e] = t < left ? (red[t] + red[3 * GT + t]) + (red[GT + t] + red[4 * GT + t]) : 0.f;
                    k[e] = kin[e] = t < left ? red[2 * GT + t] + red[5 * GT + t] : 0.f;
#pragma unroll
                    for (int o = 1; o < 32; o *= 2) {
                        const float x = __shfl_down_sync(~0u, v[e], o), y = __shfl_up_sync(~0u, kin[e], o);
                        if (lane + o < 32) v[e] += x;       // from this token on
                        if (lane >= o) kin[e] += y;         // up to this token
                    }
                }
                total = (dots[0] + dots[1]) * ga[GT - 1];
                const float later = __shfl_sync(~0u, v[1], 0), earlier = __shfl_sync(~0u, kin[0], 31);
                const float dg[2] = {total + (kin[0] - k[0]) + (v[0] + later), total + (earlier + kin[1] - k[1]) + v[1]};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    if (t < left) {
                        reinterpret_cast<float*>(p.dG.p)[b * p.dG.bs + h * p.dG.hs + (tok + t) * p.dG.ts] = dg[e];
                        reinterpret_cast<float*>(p.dBeta.p)[b * p.dBeta.bs + h * p.dBeta.hs + (tok + t) * p.dBeta.ts] = dbe[t];
                    }
                }
            }
        }
    }
    __syncthreads();
    if (warp == 9) tmem_dealloc(ctl.tmem, 512);
}

// dQ, dK [B][hk][N][dk] (strided views; half of the grid each) = the sums over the r value heads of a key head of the fp32
// [B][h][N][dk] partial gradients, in head order.
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
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(out.p) + b * out.bs + kh * out.hs + t * out.ts + c) =
        make_uint2(pack2(a.x, a.y), pack2(a.z, a.w));
}
