// gemm_fp8.hip - fp8 e4m3 products with a binary32 scale per block of 128 along
// K, dense, over a mixture's experts, and the experts' weight gradients.
//
//   C[i][j] = sum over blocks g of  sa[g][i] * sb[g][j / b] * P_g[i][j],
//   P_g[i][j] = sum over k in block g of a[i][k] * b[j][k]
//
// A is M x K and B is N x K, both with K contiguous.  Binary32 scales are no
// powers of two, so the matrix unit computes P_g unscaled from zero and each P_g
// is added to the binary32 accumulator with the product of its scales, one FMA
// per element.  The operands' K order inside a block is free as long as both use
// the same one.
//
// Two ways to compute P_g of a 16 x 16 tile:
//   - one 16x16x128 fp8 MFMA.  Inside each group of 8 consecutive k its adder cuts
//     every product towards zero at 2^-13 of the group's largest (exactly so:
//     tests/test_gpu_fp8_unit.py; across groups all 24 bits survive): an error of
//     1.4e-5 of the result's norm on normal values, 2.9e-5 with a few columns 16 times
//     the others.  Rounding the result is 120 (bf16, 1.7e-3) or 15 (f16, 2.1e-4) times
//     coarser, so the tiled kernel takes it for outputs of 16 bits.  The error goes
//     with the products' magnitudes, not with the value: an element whose terms
//     cancel may lose more than its own rounding (an F32 output does not).
//   - EXACT: both operands widened to binary16 (every e4m3 value is one) and four
//     chained 16x16x32 binary16 MFMAs, whose products are exact and whose sums are
//     kept in binary32, at half the rate: for binary32 outputs, and everywhere in
//     the streaming kernel, whose time is that of reading B.
//
// Measured (MI355X; a copy reaches 5.0 TB/s, large library products 2.84 PFLOP/s in
// fp8 and 1.44 in bfloat16): 4096^3 to bf16 61.5 us (2.24 PFLOP/s) and to f32 114-126
// us; 8192 rows over 8 experts of 4096 x 4096 155-182 us as the rows fall; their
// weight gradients (2048 x 4096, f32) 165 us, of which writing 268 MB is 54; 32 rows
// over 8 experts 20.8-26.3 us (5.1 TB/s of weights at 26.3); one token through 4096 x
// 4096 6.2 us.
#include "gemm_tiled.h"
#include "launch.h"
#include "moe_args.h"

namespace dg {

// (the unscaled form: both scale operands the constant 0)
DG_DEV floatx4 mfma_fp8(u32x8 b, u32x8 a, floatx4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(intx8, b), __builtin_bit_cast(intx8, a),
                                                            c, 0, 0, 0, 0, 0, 0);
}

// A lane's 32 e4m3 values widened to binary16.
struct Wide {
    half8 v[4];
};
DG_DEV half8 widen8(unsigned lo, unsigned hi)
{
    const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return half8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
template <bool EXACT>
DG_DEV auto operand(u32x8 q)
{
    if constexpr (EXACT)
        return Wide{{widen8(q[0], q[1]), widen8(q[2], q[3]), widen8(q[4], q[5]), widen8(q[6], q[7])}};
    else
        return q;
}
DG_DEV floatx4 block_product(u32x8 b, u32x8 a) { return mfma_fp8(b, a, floatx4{0.f, 0.f, 0.f, 0.f}); }
DG_DEV floatx4 block_product(const Wide &b, const Wide &a)
{
    floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[q], a.v[q], c, 0, 0, 0);
    return c;
}

// A 16-byte chunk whose first byte is value k: the bytes at or past kend cleared.
DG_DEV u32x4 keep_bytes(u32x4 v, int k, int kend)
{
    const int n = kend - k;   // valid bytes, any sign
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int b = n - 4 * d;
        v[d] &= b >= 4 ? ~0u : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
    }
    return v;
}

// ------------------------------------------------------- segments of experts
// Offsets come from device memory: they are clamped to [0, rows], so whatever
// they hold, every access stays inside the operands.
DG_DEV void seg_bounds(const int32_t *off, int e, int experts, int rows, int &lo, int &hi)
{
    lo = hi = 0;
    if (e < experts) {
        lo = min(max(off[e], 0), rows);
        hi = max(lo, min(max(off[e + 1], 0), rows));
    }
}
DG_DEV int wave_scan(int v)   // inclusive sum over the lanes
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}
// Row tiles of bm rows over all segments, at most `most`.
DG_DEV int seg_total(const int32_t *off, int experts, int rows, int bm, int most)
{
    int64_t total = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        int lo, hi;
        seg_bounds(off, e0 + (threadIdx.x & 63), experts, rows, lo, hi);
        total += __builtin_amdgcn_readlane(wave_scan((hi - lo + bm - 1) / bm), 63);
    }
    return (int)(total < most ? total : most);
}
// Row tile t: its expert, its first row and the end of the expert's rows.
DG_DEV void seg_find(const int32_t *off, int experts, int rows, int bm, int t, int &e, int &row0, int &end)
{
    int base = 0;
    e = 0, row0 = 0, end = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        int lo, hi;
        seg_bounds(off, e0 + (threadIdx.x & 63), experts, rows, lo, hi);
        const int n = (hi - lo + bm - 1) / bm, incl = wave_scan(n);
        const unsigned long long past = __ballot(base + incl > t);
        if (past) {
            const int f = __builtin_ctzll(past);
            e = e0 + f;
            const int first = base + __builtin_amdgcn_readlane(incl, f) - __builtin_amdgcn_readlane(n, f);
            row0 = __builtin_amdgcn_readlane(lo, f) + (t - first) * bm;
            end = __builtin_amdgcn_readlane(hi, f);
            return;
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
}

// ---------------------------------------------------------------- tiled kernel
// What bounds it (256 x 256, 4096^3): a step of 128 takes 1.56 us where its MFMAs
// take 0.94 at the clock it ran at (2.17 GHz, counters: matrix unit 56 % busy while
// the CU is, no LDS conflicts to speak of).  In timing copies the step took 1.29 us
// without the loads, 1.37 without the scaling FMAs and 1.12 without both: the three
// share the issue of two waves per SIMD.  Four MFMAs and then sixteen FMAs, or
// pairs, were 5 % slower than one MFMA and four FMAs at a time.
// One workgroup computes a BM x BN tile; its waves share the tile as WM x WN.
// Operand blocks go from memory straight to LDS, one stage per block of 128, and
// the loads of the next stages run under the current one's MFMAs.  A stage holds
// each operand as rows of 128 bytes with the 16-byte chunk index XORed with
// (row >> 1) & 7: a load reads 8 whole lines, and the 16 rows of a fragment read
// lie in 16 different chunks of the LDS banks.  Then come the rows' scales of A and
// of B (one per column: a shared scale is spread here, by the load's addresses).
template <int BM, int BN, int WM, int WN, int NBUF, int MODE, bool BB1, bool EXACT>
__global__ void __launch_bounds__(WM *WN * 64, 2) fp8_tiled_kernel(Fp8Args p)
{
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    static_assert(128 % WTN == 0, "a wave's columns lie in one scale block");
    constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    constexpr int STAGE = A_BYTES + B_BYTES + (BM + BN) * 4;
    static_assert(STAGE % 256 == 0, "stage alignment");
    constexpr int A_LD = BM / 8 / NW, B_LD = BN / 8 / NW;       // 1 KB loads per wave and stage
    static_assert(A_LD * NW * 8 == BM && B_LD * NW * 8 == BN, "whole loads");
    constexpr int S_NL = (BM + BN) / 64;                        // 256-byte scale loads per stage
    constexpr int S_LD = (S_NL + NW - 1) / NW;                  // (waves past the last one repeat it: no branch)
    constexpr int LPS = A_LD + B_LD + S_LD;                     // loads a wave issues per stage
    constexpr int RP = WTN + 4;                                 // row pitch of the output staging
    constexpr int LDS_BYTES = NBUF * STAGE > NW * 16 * RP * 4 ? NBUF * STAGE : NW * 16 * RP * 4;
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int L16 = lane & 15, g16 = lane >> 4;

    // ---- the tile: consecutive workgroups of a die take consecutive tiles, four
    // row tiles side by side (over experts the next four in the list of all row
    // tiles, which may belong to two experts)
    int m0, mend, n0, expert = 0, kbeg = 0, kend = p.K;
    {
        int T, t, e_rows = p.tiles_m;
        if constexpr (MODE == FP8_ROWS) {
            e_rows = seg_total(p.off, p.experts, p.M, BM, p.tiles_m);
            T = e_rows * p.tiles_n;
            if ((int)blockIdx.x >= T) return;
            t = xcd_remap(blockIdx.x, T);
        } else if constexpr (MODE == FP8_WGRAD) {
            // every die gets an eighth of each expert's tiles (an expert's K is its
            // rows: a die with one whole expert would wait for the longest)
            T = p.tiles_m * p.tiles_n;
            const int pad = (T + 7) & ~7;
            expert = blockIdx.x / pad;
            const int i = blockIdx.x - expert * pad;
            if (i >= T) return;
            t = xcd_remap(i, T);
        } else {
            T = p.tiles_m * p.tiles_n;
            t = xcd_remap(blockIdx.x, T);
        }
        const int per = 4 * p.tiles_n, grp = t / per, gm = min(e_rows - grp * 4, 4), tl = t - grp * per;
        const int tm = grp * 4 + tl % gm;
        n0 = tl / gm * BN;
        if constexpr (MODE == FP8_ROWS) {
            seg_find(p.off, p.experts, p.M, BM, tm, expert, m0, mend);
        } else {
            m0 = tm * BM;
            mend = p.M;
        }
        if constexpr (MODE == FP8_WGRAD) {
            int lo, hi;
            seg_bounds(p.off, expert, p.experts, p.K, lo, hi);
            kbeg = lo & ~(FP8_BLOCK - 1);   // segments start on whole scale blocks
            kend = hi > lo ? hi : kbeg;
        }
        if constexpr (MODE == FP8_DENSE) {
            kbeg = blockIdx.y * p.k_slice;
            kend = min(p.K, kbeg + p.k_slice);
        }
    }
    // (the same in every lane: in scalar registers, as the buffer descriptors need them)
    for (int *v : {&m0, &mend, &n0, &expert, &kbeg, &kend}) *v = __builtin_amdgcn_readfirstlane(*v);
    const int rows = min(mend - m0, BM), cols = min(p.N - n0, BN);
    const int nsteps = (kend - kbeg + FP8_BLOCK - 1) / FP8_BLOCK;

    // Each die starts at another block and goes round (the last block, which may be
    // short, stays last): rows of a pitch of whole kilobytes keep one block of all
    // of them in few memory channels, where dies that walk K in step meet (32 rows
    // over 8 experts of 4096 x 4096, 128 x 128 tiles, 38.6 -> 34.9 us; weight
    // gradients 177 -> 174).  The 256 x 256 tile loses 2 % by it.
    int turn = 0;
    if constexpr (BM < 256)
        if (nsteps > 1) turn = (int)(blockIdx.x & 7) * ((nsteps + 7) / 8) % (nsteps - 1);

    // ---- operands from the tile's origin; extents in bytes up to the end of the
    // last row's last chunk (rows are readable to their next 16-byte boundary)
    const char *Ab = reinterpret_cast<const char *>(p.A) + (int64_t)m0 * p.lda + kbeg;
    const char *Bb = reinterpret_cast<const char *>(p.B) + (int64_t)n0 * p.ldb + kbeg;
    const float *Sa = p.sa + (int64_t)(kbeg / FP8_BLOCK) * p.ld_sa + m0;
    const float *Sb = p.sb + (int64_t)(kbeg / FP8_BLOCK) * p.ld_sb + (BB1 ? n0 : n0 / FP8_BLOCK);
    if constexpr (MODE == FP8_ROWS) {
        Bb += (int64_t)expert * p.stride_b;
        Sb += (int64_t)expert * p.stride_sb;
    }
    const uint32_t kbytes = (uint32_t)((kend - kbeg + 15) & ~15);
    const uint32_t a_ext = (uint32_t)(rows - 1) * (uint32_t)p.lda + kbytes;
    const uint32_t b_ext = (uint32_t)(cols - 1) * (uint32_t)p.ldb + kbytes;
    const uint32_t sa_ext = (uint32_t)rows * 4;
    const uint32_t sb_ext = BB1 ? (uint32_t)cols * 4
                                : (uint32_t)((n0 + cols - 1) / FP8_BLOCK - n0 / FP8_BLOCK + 1) * 4;
    // lane l of load q writes chunk position l & 7 of row q * 8 + l / 8
    uint32_t oa[A_LD], ob[B_LD], os[S_LD];
#pragma unroll
    for (int i = 0; i < A_LD; ++i) {
        const int r = (i * NW + wave) * 8 + (lane >> 3);
        oa[i] = (uint32_t)r * (uint32_t)p.lda + (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) * 16;
    }
#pragma unroll
    for (int i = 0; i < B_LD; ++i) {
        const int r = (i * NW + wave) * 8 + (lane >> 3);
        ob[i] = (uint32_t)r * (uint32_t)p.ldb + (uint32_t)((lane & 7) ^ ((r >> 1) & 7)) * 16;
    }
#pragma unroll
    for (int i = 0; i < S_LD; ++i) {
        const int r = (i * NW + wave) % S_NL * 64 + lane;   // rows of A, then columns of B
        os[i] = r < BM ? r * 4 : (BB1 ? (r - BM) * 4 : ((n0 + r - BM) / FP8_BLOCK - n0 / FP8_BLOCK) * 4);
    }
    // Load i of step j into stage j % NBUF.  Past the last step the ranges are empty
    // (zeros into a stage nobody reads): every wave's count of loads in flight
    // stays the same.
    auto load_one = [&](int j, int i) {
        const bool real = j < nsteps;
        int g = j + turn;   // the block of step j
        g = j >= nsteps - 1 ? j : (g >= nsteps - 1 ? g - (nsteps - 1) : g);
        const int64_t k = real ? (int64_t)g * FP8_BLOCK : 0;
        char *sb = smem + (j % NBUF) * STAGE;
        if (i < A_LD) {
            buf_ld16_lds(make_rsrc(Ab + k, real ? a_ext - (uint32_t)k : 0u), oa[i], sb + (i * NW + wave) * 1024);
        } else if (i < A_LD + B_LD) {
            buf_ld16_lds(make_rsrc(Bb + k, real ? b_ext - (uint32_t)k : 0u), ob[i - A_LD],
                         sb + A_BYTES + ((i - A_LD) * NW + wave) * 1024);
        } else {
            const int q = ((i - A_LD - B_LD) * NW + wave) % S_NL;   // wave-uniform
            const bool ofa = q < BM / 64;
            const float *base = ofa ? Sa + (real ? g : 0) * p.ld_sa : Sb + (real ? g : 0) * p.ld_sb;
            buf_ld4_lds(make_rsrc(base, real ? (ofa ? sa_ext : sb_ext) : 0u), os[i - A_LD - B_LD],
                        sb + A_BYTES + B_BYTES + q * 256);
        }
    };
    auto load_stage = [&](int j) {
#pragma unroll
        for (int i = 0; i < LPS; ++i) load_one(j, i);
    };

    floatx4 acc[FM][FN];
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
        for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = floatx4{0.f, 0.f, 0.f, 0.f};

    // this lane's chunks (k 16 g16 .. +15 and 64 more) of a 16-row fragment
    const int flo = L16 * 128 + ((g16 ^ (L16 >> 1)) << 4), fhi = flo ^ 64;
    auto frag = [&](const char *base) {
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(base + flo);
        const u32x4 hi = *reinterpret_cast<const u32x4 *>(base + fhi);
        return u32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };
    auto mask = [&](u32x8 v, int k) {   // k: the block's first value
        const u32x4 lo = keep_bytes(u32x4{v[0], v[1], v[2], v[3]}, k + g16 * 16, kend);
        const u32x4 hi = keep_bytes(u32x4{v[4], v[5], v[6], v[7]}, k + 64 + g16 * 16, kend);
        return u32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };
    // One step: the MFMAs row of tiles by row of tiles, the scaling FMAs of a tile QD
    // MFMAs after its own, and A's next fragment read under the present
    // row.  All reads of stage st are issued before its last row, so the one barrier
    // of the step comes there: it finds stage st + 1 landed and frees stage st's
    // buffer for the loads of stage st + NBUF, and the last row's MFMAs cover the
    // first reads of stage st + 1.
    using Op = decltype(operand<EXACT>(u32x8{}));
    constexpr int D = FM >= 4 ? 2 : 1, R = 2 * D;   // rows read ahead, fragments held
    static_assert(FM % R == 0, "the ring starts over with each step");
    u32x8 a[R], braw[2];
    Op b[FN];
    float sa[R];      // scales of the rows of tiles in hand
    floatx4 sb[FN];   // BB1: the columns' scales; else sb[0][0], the block's
    const char *const sA0 = smem + wm * WTM * 128, *const sB0 = smem + A_BYTES + wn * WTN * 128;
    const float *const scA0 = reinterpret_cast<const float *>(smem + A_BYTES + B_BYTES) + wm * WTM + L16;
    const float *const scB0 = reinterpret_cast<const float *>(smem + A_BYTES + B_BYTES) + BM + wn * WTN;
    auto read_a = [&](int st, int mi) {
        const int o = (st % NBUF) * STAGE;
        a[mi % R] = frag(sA0 + o + mi * 2048);
        sa[mi % R] = scA0[o / 4 + mi * 16];
    };
    auto read_b = [&](int st, int ni) { return frag(sB0 + (st % NBUF) * STAGE + ni * 2048); };
    auto read_sb = [&](int st) {
        const float *sc = scB0 + (st % NBUF) * STAGE / 4;
        if constexpr (BB1) {
#pragma unroll
            for (int ni = 0; ni < FN; ++ni) sb[ni] = *reinterpret_cast<const floatx4 *>(sc + ni * 16 + g16 * 4);
        } else {
            sb[0][0] = sc[0];
        }
    };
    constexpr int QD = FM * FN > 16 ? 2 : 3;
    auto step = [&](int st, auto last_tag) {
        constexpr bool LAST = decltype(last_tag)::value;
        floatx4 q[QD + 1];
        float s[2];
        auto scale_add = [&](int t) {
            const int mi = t / FN, ni = t % FN;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[mi][ni][e] = __builtin_fmaf(q[t % (QD + 1)][e], BB1 ? s[mi & 1] * sb[ni][e] : s[mi & 1], acc[mi][ni][e]);
        };
        if constexpr (LAST) {   // bytes past K may hold anything, NaN codes too
            const int k = kbeg + st * FP8_BLOCK;
#pragma unroll
            for (int ni = 0; ni < FN; ++ni) b[ni] = operand<EXACT>(mask(read_b(st, ni), k));
        } else if constexpr (EXACT) {
            b[FN - 1] = operand<EXACT>(braw[(FN - 1) & 1]);
        }
#pragma unroll
        for (int mi = 0; mi < FM; ++mi) {
            if constexpr (!LAST) {
                if (mi == FM - D) {
                    wait_vm_barrier<(NBUF - 2) * LPS>();
                }
            }
            if constexpr (LAST) a[mi % R] = mask(a[mi % R], kbeg + st * FP8_BLOCK);
            s[mi & 1] = BB1 ? sa[mi % R] : sa[mi % R] * sb[0][0];
            const Op aw = operand<EXACT>(a[mi % R]);
            if (mi < FM - D) read_a(st, mi + D);
            else if (!LAST) read_a(st + 1, mi + D - FM);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ni = 0; ni < FN; ++ni) {
                const int t = mi * FN + ni;
                q[t % (QD + 1)] = block_product(b[ni], aw);
                __builtin_amdgcn_sched_barrier(0);
                if (!LAST && mi == FM - 1) {
                    if constexpr (EXACT) {
                        if (ni > 0) b[ni - 1] = operand<EXACT>(braw[(ni - 1) & 1]);
                        braw[ni & 1] = read_b(st + 1, ni);
                    } else {
                        b[ni] = read_b(st + 1, ni);
                    }
                }
                if constexpr (!LAST) {   // the loads, spread over the MFMAs after the barrier
#pragma unroll
                    for (int i = 0; i < LPS; ++i)
                        if (t - (FM - D) * FN == i * D * FN / LPS) load_one(st + NBUF, i);
                }
                if (t >= QD) scale_add(t - QD);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int t = FM * FN - QD; t < FM * FN; ++t) scale_add(t);
        if constexpr (!LAST) read_sb(st + 1);
    };
    if (nsteps > 0) {
#pragma unroll
        for (int j = 0; j < NBUF; ++j) load_stage(j);
        wait_vm_barrier<(NBUF - 1) * LPS>();
        if (wm * WTM < rows) {
#pragma unroll
            for (int mi = 0; mi < D; ++mi) read_a(0, mi);
            read_sb(0);
            if (nsteps > 1) {
#pragma unroll
                for (int ni = 0; ni < FN; ++ni) {
                    if constexpr (EXACT) {
                        braw[ni & 1] = read_b(0, ni);
                        if (ni < FN - 1) b[ni] = operand<EXACT>(braw[ni & 1]);
                    } else {
                        b[ni] = read_b(0, ni);
                    }
                }
            }
            for (int st = 0; st < nsteps - 1; ++st) step(st, std::false_type{});
            step(nsteps - 1, std::true_type{});
        } else {   // no rows for this wave: its share of the loads, and the barriers
            for (int st = 0; st < nsteps - 1; ++st) {
                wait_vm_barrier<(NBUF - 2) * LPS>();
                load_stage(st + NBUF);
            }
        }
    }

    // ---- output: lane l of a 16 x 16 tile holds row l & 15 and columns
    // 4 (l >> 4) .. +3; 16 rows at a time go through LDS to be stored by rows.
    __syncthreads();   // (waits for the empty loads too)
    char *Cp = reinterpret_cast<char *>(p.C);
    int64_t ldc = p.ldc;
    int type = p.out_type;
    if constexpr (MODE == FP8_DENSE) {
        if (p.split_k > 1) {
            Cp = reinterpret_cast<char *>(p.ws + (int64_t)blockIdx.y * p.M * p.N);
            ldc = p.N;
            type = T_F32;
        }
    }
    const int esz = type == T_F32 ? 4 : 2;
    Cp += ((MODE == FP8_WGRAD ? expert * p.stride_c : 0) + (int64_t)m0 * ldc + n0) * esz;
    float *sE = reinterpret_cast<float *>(smem) + wave * 16 * RP;
    const bool vec = ((uintptr_t)Cp & 15) == 0 && (ldc * esz & 15) == 0;
#pragma unroll
    for (int mi = 0; mi < FM; ++mi) {
#pragma unroll
        for (int ni = 0; ni < FN; ++ni)
            *reinterpret_cast<floatx4 *>(sE + L16 * RP + ni * 16 + g16 * 4) = acc[mi][ni];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const int r0 = wm * WTM + mi * 16;
        if (type == T_F32) {
            constexpr int LPR = WTN / 4, RPI = 64 / LPR;
            const int c = lane % LPR * 4, col = wn * WTN + c;
#pragma unroll
            for (int it = 0; it < 16 / RPI; ++it) {
                const int rr = it * RPI + lane / LPR, row = r0 + rr;
                if (row >= rows || col >= cols) continue;
                const floatx4 v = *reinterpret_cast<const floatx4 *>(sE + rr * RP + c);
                const int64_t idx = (int64_t)row * ldc + col;
                if (vec && col + 4 <= cols) store4_f32(Cp, T_F32, idx, v);
                else
                    for (int e = 0; e < 4; ++e)
                        if (col + e < cols) reinterpret_cast<float *>(Cp)[idx + e] = v[e];
            }
        } else {
            constexpr int LPR = WTN / 8, RPI = 64 / LPR;
            const int c = lane % LPR * 8, col = wn * WTN + c;
#pragma unroll
            for (int it = 0; it < (16 + RPI - 1) / RPI; ++it) {
                const int rr = it * RPI + lane / LPR, row = r0 + rr;
                if (rr >= 16 || row >= rows || col >= cols) continue;
                const floatx4 lo = *reinterpret_cast<const floatx4 *>(sE + rr * RP + c);
                const floatx4 hi = *reinterpret_cast<const floatx4 *>(sE + rr * RP + c + 4);
                const int64_t idx = (int64_t)row * ldc + col;
                if (vec && col + 8 <= cols) store8_f16x(Cp, type, idx, lo, hi);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < cols) store_f32(Cp, type, idx + e, e < 4 ? lo[e & 3] : hi[e & 3]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

// ------------------------------------------------------------- streaming kernel
// Few rows: the time is that of reading B once.  A workgroup takes 16 FM rows x
// 16 FN columns and cuts K over its NW waves (wave w takes blocks w, w + NW, ...),
// operands go from memory to registers, and the waves' sums are added in wave
// order through LDS: no workspace, and the same result on every run.  One row, N = K =
// 4096: 6.2 us (2.7 TB/s, mostly latency: each wave has one batch of loads);
// 64 x 64 tiles with a K split and its sum took 3 us more.
template <int FM, int FN, int NW, int MODE, bool BB1>
__global__ void __launch_bounds__(NW * 64) fp8_stream_kernel(Fp8Args p)
{
    constexpr int BM = 16 * FM, BN = 16 * FN, T = FM * FN;
    constexpr int U = 4;   // blocks whose loads are issued together
    __shared__ floatx4 red[NW][T][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int L16 = lane & 15, g16 = lane >> 4;
    int m0, mend, n0, expert = 0;
    if constexpr (MODE == FP8_ROWS) {
        const int e_rows = seg_total(p.off, p.experts, p.M, BM, p.tiles_m);
        const int t = blockIdx.x;   // column tiles of one row tile side by side
        if (t >= e_rows * p.tiles_n) return;
        n0 = t % p.tiles_n * BN;
        seg_find(p.off, p.experts, p.M, BM, t / p.tiles_n, expert, m0, mend);
    } else {
        n0 = (int)(blockIdx.x % p.tiles_n) * BN;
        m0 = (int)(blockIdx.x / p.tiles_n) * BM;
        mend = p.M;
    }
    const int rows = min(mend - m0, BM), cols = min(p.N - n0, BN);
    // rows and columns past the tile repeat its last one and are not stored
    const char *Ap[FM], *Bp[FN];
    const float *Sa[FM], *Sb[FN];
    const int64_t eb = MODE == FP8_ROWS ? (int64_t)expert * p.stride_b : 0;
    const int64_t es = MODE == FP8_ROWS ? (int64_t)expert * p.stride_sb : 0;
#pragma unroll
    for (int mi = 0; mi < FM; ++mi) {
        const int r = m0 + min(mi * 16 + L16, rows - 1);
        Ap[mi] = reinterpret_cast<const char *>(p.A) + (int64_t)r * p.lda + g16 * 16;
        Sa[mi] = p.sa + r;
    }
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) {
        const int c = n0 + min(ni * 16 + L16, cols - 1);
        Bp[ni] = reinterpret_cast<const char *>(p.B) + eb + (int64_t)c * p.ldb + g16 * 16;
        Sb[ni] = p.sb + es + (BB1 ? n0 + ni * 16 + g16 * 4 : n0 / FP8_BLOCK);
    }
    floatx4 acc[FM][FN];
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
        for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int nb = (p.K + FP8_BLOCK - 1) / FP8_BLOCK, whole = p.K / FP8_BLOCK;
    auto load = [&](const char *q, int b, bool nt) {
        const int k = b * FP8_BLOCK;
        u32x4 lo = u32x4{0u, 0u, 0u, 0u}, hi = lo;
        if (b < whole) {
            lo = nt ? ld16_nt(q + k) : ld16(q + k);
            hi = nt ? ld16_nt(q + k + 64) : ld16(q + k + 64);
        } else if (b < nb) {   // the chunks that hold values, and of those the bytes below K
            if (k + g16 * 16 < p.K) lo = keep_bytes(ld16(q + k), k + g16 * 16, p.K);
            if (k + 64 + g16 * 16 < p.K) hi = keep_bytes(ld16(q + k + 64), k + 64 + g16 * 16, p.K);
        }
        return u32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };
    for (int b0 = wave; b0 < nb; b0 += NW * U) {
        u32x8 a[U][FM], b[U][FN];
        float sa[U][FM];
        floatx4 sb[U][FN];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int bb = b0 + u * NW, bs = min(bb, nb - 1);
#pragma unroll
            for (int ni = 0; ni < FN; ++ni) {
                b[u][ni] = load(Bp[ni], bb, true);
                const float *s = Sb[ni] + (int64_t)bs * p.ld_sb;
                if constexpr (BB1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) sb[u][ni][e] = s[min(e, p.N - 1 - (n0 + ni * 16 + g16 * 4))];
                } else {
                    sb[u][ni][0] = s[0];
                }
            }
#pragma unroll
            for (int mi = 0; mi < FM; ++mi) {
                a[u][mi] = load(Ap[mi], bb, false);
                sa[u][mi] = Sa[mi][(int64_t)bs * p.ld_sa];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u * NW >= nb) break;
            Wide bw[FN];
#pragma unroll
            for (int ni = 0; ni < FN; ++ni) bw[ni] = operand<true>(b[u][ni]);
#pragma unroll
            for (int mi = 0; mi < FM; ++mi) {
                const Wide aw = operand<true>(a[u][mi]);
#pragma unroll
                for (int ni = 0; ni < FN; ++ni) {
                    const floatx4 q = block_product(bw[ni], aw);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[mi][ni][e] = __builtin_fmaf(q[e], sa[u][mi] * sb[u][ni][BB1 ? e : 0], acc[mi][ni][e]);
                }
            }
        }
    }
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
        for (int ni = 0; ni < FN; ++ni) red[wave][mi * FN + ni][lane] = acc[mi][ni];
    __syncthreads();
    for (int u = threadIdx.x; u < T * 64; u += NW * 64) {
        const int t = u >> 6, l = u & 63;
        floatx4 v = red[0][t][l];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += red[w][t][l];
        const int row = t / FN * 16 + (l & 15), col = t % FN * 16 + (l >> 4) * 4;
        if (row >= rows) continue;
        const int64_t idx = (int64_t)(m0 + row) * p.ldc + n0 + col;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < cols) store_f32(p.C, p.out_type, idx + e, v[e]);
    }
}

// ------------------------------------------------------------------------ host
namespace {
const Fp8Shape g_shapes[FP8_KERNELS] = {
    {16, 16, 512, true, "fp8_stream_16x16"},
    {64, 64, 256, false, "fp8_tiled_64x64"},
    {128, 128, 256, false, "fp8_tiled_128x128"},
    {256, 256, 512, false, "fp8_tiled_256x256"},
};

template <int MODE, bool BB1>
const void *fp8_kernel(int kernel, bool exact)
{
    if constexpr (MODE != FP8_WGRAD) {
        if (kernel == FP8_STREAM16) return reinterpret_cast<const void *>(fp8_stream_kernel<1, 1, 8, MODE, BB1>);
    }
    if (kernel == FP8_TILE64)
        return exact ? reinterpret_cast<const void *>(fp8_tiled_kernel<64, 64, 2, 2, 3, MODE, BB1, true>)
                     : reinterpret_cast<const void *>(fp8_tiled_kernel<64, 64, 2, 2, 3, MODE, BB1, false>);
    if (kernel == FP8_TILE128)
        return exact ? reinterpret_cast<const void *>(fp8_tiled_kernel<128, 128, 2, 2, 2, MODE, BB1, true>)
                     : reinterpret_cast<const void *>(fp8_tiled_kernel<128, 128, 2, 2, 2, MODE, BB1, false>);
    if (kernel == FP8_TILE256 && !exact)
        return reinterpret_cast<const void *>(fp8_tiled_kernel<256, 256, 2, 4, 2, MODE, BB1, false>);
    return nullptr;
}
}  // namespace

const Fp8Shape &fp8_shape(int kernel) { return g_shapes[kernel]; }

hipError_t launch_fp8(int kernel, int mode, int b_block, const Fp8Args &a, hipStream_t s)
{
    if (kernel < 0 || kernel >= FP8_KERNELS) return hipErrorInvalidValue;
    const Fp8Shape &sh = g_shapes[kernel];
    const void *fn = nullptr;
    const bool exact = a.out_type == T_F32;
    if (mode == FP8_DENSE) fn = b_block == 1 ? fp8_kernel<FP8_DENSE, true>(kernel, exact) : fp8_kernel<FP8_DENSE, false>(kernel, exact);
    else if (mode == FP8_ROWS) fn = fp8_kernel<FP8_ROWS, false>(kernel, exact);
    else if (mode == FP8_WGRAD) fn = fp8_kernel<FP8_WGRAD, true>(kernel, exact);
    if (!fn) return hipErrorInvalidValue;
    Fp8Args arg = a;
    arg.tiles_n = (a.N + sh.bn - 1) / sh.bn;
    if (mode == FP8_ROWS) {
        // every expert may end inside a tile, but no tile is empty
        const int64_t most = (a.M + (int64_t)a.experts * (sh.bm - 1)) / sh.bm;
        arg.tiles_m = (int)(most < a.M ? most : a.M);
    } else {
        arg.tiles_m = (a.M + sh.bm - 1) / sh.bm;
    }
    const int64_t tiles = (int64_t)arg.tiles_m * arg.tiles_n;
    const __int128 grid = mode == FP8_WGRAD ? (__int128)((tiles + 7) / 8 * 8) * a.experts : tiles;   // (whole turns of the 8 dies per expert)
    if (grid == 0) return hipSuccess;
    if (!grid_fits(grid, sh.threads)) return hipErrorInvalidConfiguration;
    if (arg.split_k < 1 || arg.split_k > 65535) return hipErrorInvalidValue;
    void *args[] = {&arg};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)grid, (unsigned)arg.split_k, 1), dim3(sh.threads, 1, 1), args, 0, s);
    return e != hipSuccess ? e : hipGetLastError();
}

}  // namespace dg
