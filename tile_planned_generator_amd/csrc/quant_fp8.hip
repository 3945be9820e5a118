// quant_fp8.hip - 16- or 32-bit activations -> fp8 e4m3 codes with one binary32
// scale per 128 consecutive values, along the rows or down the columns: the
// operands of the block-scaled products.
//
// Per block: s = max(max |x| / 448, 2^-126), code = e4m3(x / s), nearest even.
// Both divisions are correctly rounded in binary32, so |x / s| never rounds past
// 448 and no value saturates.  A block with an infinity or a NaN follows the
// formula: s is that infinity or NaN, and x / s is NaN where it is not finite.
// Rows may be picked through an index (row r is X's row index[r] / index_div,
// zeros where the index names no row): the copy of a token's row for each of its
// experts is quantised without being written first.
#include "kcommon.h"
#include "moe_args.h"
#include "row8.h"

namespace dg {

namespace {
constexpr float kMax = 448.0f;
constexpr float kTiny = 1.17549435e-38f;   // 2^-126

// |x| as its bits: their order as whole numbers is that of the magnitudes, with
// infinities above every finite value and NaN above those, so a whole-number
// maximum keeps a NaN (one instruction where a float maximum that does takes four).
DG_DEV unsigned mag_bits(float x) { return __builtin_bit_cast(unsigned, x) & 0x7fffffffu; }
DG_DEV unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

// The divisor of a block: x / s as q = x r, q + (x - q s) r with r = 1/s rounded
// is the correctly rounded quotient as long as nothing underflows (Markstein's
// theorem), which holds for every x whose code is not zero when s is at least
// 2^-90; smaller and non-finite scales take the division itself (r = 0).
struct Scale {
    float s, r;
    Scale() = default;
    DG_DEV explicit Scale(unsigned amax)
    {
        s = __fdiv_rn(__builtin_bit_cast(float, amax), kMax);
        s = s < kTiny ? kTiny : s;
        r = s >= 8.0779356694631609e-28f && s < __builtin_inff() ? __fdiv_rn(1.0f, s) : 0.f;   // 2^-90
    }
    DG_DEV bool plain() const { return r == 0.f; }
    template <bool PLAIN>
    DG_DEV float quotient(float x) const
    {
        if (PLAIN) return __fdiv_rn(x, s);
        const float q = x * r;
        return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
    }
};

// four codes, the first in the low byte
template <bool PLAIN>
DG_DEV unsigned codes4(const Scale &sc, float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(sc.quotient<PLAIN>(a), sc.quotient<PLAIN>(b), 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(sc.quotient<PLAIN>(c), sc.quotient<PLAIN>(d), w, true);
}

// the value of another lane of the same 16 (rotated by N) or of the same four (lane N)
template <int N>
DG_DEV unsigned ror16(unsigned v) { return (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xf, 0xf, true); }
template <int N>
DG_DEV float quad_lane(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), N * 0x55, 0xf, 0xf, true));
}

// The N rows first .. first+N-1 at column c, eight values of each: all their indices
// are loaded, then all their values.
template <int N, typename T>
DG_DEV void load_rows(const QuantFp8Args &p, int64_t first, int c, floatx8 (&v)[N])
{
    int64_t t[N];
    if (p.index) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t r = first + i;
            t[i] = p.index[r < p.rows ? r : p.rows - 1];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = t[i] < 0 ? -1 : (int64_t)((uint32_t)t[i] / (uint32_t)p.index_div);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = first + i;
    }
    typename Row8<T>::vec raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool live = first + i < p.rows && t[i] >= 0 && t[i] < p.x_rows;
        raw[i] = ld8(reinterpret_cast<const T *>(p.X) + t[i] * p.ldx + c, live ? p.cols - c : 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wide8<T>(raw[i]);
}
}  // namespace

// ------------------------------------------------------------------ along rows
// A workgroup takes 16 rows x 512 columns: wave w rows 4w .. 4w+3, 16 lanes per
// block of 128, 8 values per lane.  The scales go through LDS to be written 16
// rows at a time.  Bound by memory: 16384 rows picked from 8192 x 4096 bf16 take 30.7
// us (136 MB that it cannot do without, 4.4 TB/s), 42 before the loads of a wave's
// rows were all issued ahead of their conversions and its scales shared by lanes.
constexpr int QR_ROWS = 16, QR_COLS = 512;

template <typename T>
__global__ void __launch_bounds__(256) quant_fp8_rows_kernel(QuantFp8Args p)
{
    __shared__ float s_sc[4][QR_ROWS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int ct = (p.cols + QR_COLS - 1) / QR_COLS;
    const int64_t r0 = (int64_t)(blockIdx.x / ct) * QR_ROWS;
    const int c0 = (int)(blockIdx.x % ct) * QR_COLS, c = c0 + lane * 8;
    const bool qvec = aligned_to(p.codes, 8) && (p.ldq & 7) == 0;
    floatx8 v[4];
    load_rows<4, T>(p, r0 + wave * 4, c, v);
    // the four rows' maxima over the block's 16 lanes; lane l of each four then
    // derives the scale of row l & 3 and the others take it from there
    unsigned m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m[i] = umax(mag_bits(v[i][e]), m[i]);
        m[i] = umax(m[i], ror16<8>(m[i]));
        m[i] = umax(m[i], ror16<4>(m[i]));
        m[i] = umax(m[i], ror16<2>(m[i]));
        m[i] = umax(m[i], ror16<1>(m[i]));
    }
    const int mine = lane & 3;
    const Scale own(mine == 0 ? m[0] : mine == 1 ? m[1] : mine == 2 ? m[2] : m[3]);
    if ((lane & 15) < 4) s_sc[lane >> 4][wave * 4 + mine] = own.s;
    Scale sc[4];
    sc[0].s = quad_lane<0>(own.s), sc[0].r = quad_lane<0>(own.r);
    sc[1].s = quad_lane<1>(own.s), sc[1].r = quad_lane<1>(own.r);
    sc[2].s = quad_lane<2>(own.s), sc[2].r = quad_lane<2>(own.r);
    sc[3].s = quad_lane<3>(own.s), sc[3].r = quad_lane<3>(own.r);
    u32x2 q[4];
    if (__ballot(own.plain())) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = u32x2{codes4<true>(sc[i], v[i][0], v[i][1], v[i][2], v[i][3]),
                         codes4<true>(sc[i], v[i][4], v[i][5], v[i][6], v[i][7])};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = u32x2{codes4<false>(sc[i], v[i][0], v[i][1], v[i][2], v[i][3]),
                         codes4<false>(sc[i], v[i][4], v[i][5], v[i][6], v[i][7])};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + wave * 4 + i;
        if (r >= p.rows || c >= p.cols) continue;
        uint8_t *o = reinterpret_cast<uint8_t *>(p.codes) + r * p.ldq + c;
        if (qvec && c + 8 <= p.cols) *reinterpret_cast<u32x2 *>(o) = q[i];
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < p.cols) o[e] = (uint8_t)(q[i][e >> 2] >> (8 * (e & 3)));
    }
    __syncthreads();
    const int b = threadIdx.x / QR_ROWS, rr = threadIdx.x % QR_ROWS;
    if (b < 4 && c0 + b * FP8_BLOCK < p.cols && r0 + rr < p.rows)
        p.scales[(int64_t)(c0 / FP8_BLOCK + b) * p.ld_scale + r0 + rr] = s_sc[b][rr];
}

// ---------------------------------------------------------------- down columns
// The codes come out transposed, [cols][rows].  A workgroup takes one block of
// 128 rows x 64 columns: thread t holds rows 4 (t / 8) .. +3 of columns
// 8 (t % 8) .. +7, the columns' maxima meet in LDS, and the codes cross through
// LDS (four rows a dword) to leave as 16 bytes along the rows.  9001 x 2056 f16 take
// 18.2 us (56 MB, 3.1 TB/s): 128-byte pieces of rows in and of columns out, and four
// barriers in a workgroup that lives for one block (26.6 us before the maxima and
// scales were spread over the threads).
constexpr int QC_COLS = 64, QC_PITCH = 33;   // dwords per column: neighbouring columns in other banks

template <typename T>
__global__ void __launch_bounds__(256) quant_fp8_cols_kernel(QuantFp8Args p)
{
    __shared__ unsigned s_max[32][QC_COLS + 1];
    __shared__ unsigned s_amax[QC_COLS];
    __shared__ float s_s[QC_COLS], s_r[QC_COLS];
    __shared__ int s_plain;
    __shared__ unsigned s_q[QC_COLS * QC_PITCH];
    const int tid = threadIdx.x, cg = tid & 7, rg = tid >> 3;
    const int ct = (p.cols + QC_COLS - 1) / QC_COLS;
    const int64_t rb = blockIdx.x / ct, r0 = rb * FP8_BLOCK;
    const int c0 = (int)(blockIdx.x % ct) * QC_COLS, c = c0 + cg * 8;
    floatx8 v[4];
    if (tid < QC_COLS) s_amax[tid] = 0;
    if (tid == 0) s_plain = 0;
    load_rows<4, T>(p, r0 + rg * 4, c, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s_max[rg][cg * 8 + e] = umax(umax(mag_bits(v[0][e]), mag_bits(v[1][e])), umax(mag_bits(v[2][e]), mag_bits(v[3][e])));
    __syncthreads();
    {   // each wave takes 8 of the 32 partial maxima of every column
        const int col = tid & 63, part = tid >> 6;
        unsigned a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = umax(s_max[part * 8 + i][col], a);
        atomicMax(&s_amax[col], a);
    }
    __syncthreads();
    if (tid < QC_COLS) {
        const Scale sc(s_amax[tid]);
        s_s[tid] = sc.s, s_r[tid] = sc.r;
        if (c0 + tid < p.cols) p.scales[rb * p.ld_scale + c0 + tid] = sc.s;
        if (__ballot(sc.plain()) && tid == 0) s_plain = 1;
    }
    __syncthreads();
    const bool slow = s_plain != 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        Scale sc;
        sc.s = s_s[cg * 8 + e], sc.r = s_r[cg * 8 + e];
        s_q[(cg * 8 + e) * QC_PITCH + rg] = slow ? codes4<true>(sc, v[0][e], v[1][e], v[2][e], v[3][e])
                                                 : codes4<false>(sc, v[0][e], v[1][e], v[2][e], v[3][e]);
    }
    __syncthreads();
    const bool qvec = aligned_to(p.codes, 16) && (p.ldq & 15) == 0;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int col = it * 32 + (tid >> 3), ch = (tid & 7) * 4;   // 16 rows: 4 dwords
        const int64_t r = r0 + ch * 4;
        if (c0 + col >= p.cols || r >= p.rows) continue;
        const unsigned *q = s_q + col * QC_PITCH + ch;
        uint8_t *o = reinterpret_cast<uint8_t *>(p.codes) + (int64_t)(c0 + col) * p.ldq + r;
        if (qvec && r + 16 <= p.rows) *reinterpret_cast<u32x4 *>(o) = u32x4{q[0], q[1], q[2], q[3]};
        else
            for (int e = 0; e < 16; ++e)
                if (r + e < p.rows) o[e] = (uint8_t)(q[e >> 2] >> (8 * (e & 3)));
    }
}

hipError_t launch_quant_fp8(const QuantFp8Args &a, bool transpose, hipStream_t s)
{
    const int64_t grid = transpose ? ((int64_t)a.rows + FP8_BLOCK - 1) / FP8_BLOCK * ((a.cols + QC_COLS - 1) / QC_COLS)
                                   : ((int64_t)a.rows + QR_ROWS - 1) / QR_ROWS * ((a.cols + QR_COLS - 1) / QR_COLS);
    if (grid == 0) return hipSuccess;
    if (!grid_fits(grid, 256)) return hipErrorInvalidConfiguration;
    const void *fn;
    if (a.x_type == T_F16) fn = transpose ? (const void *)quant_fp8_cols_kernel<_Float16> : (const void *)quant_fp8_rows_kernel<_Float16>;
    else if (a.x_type == T_BF16) fn = transpose ? (const void *)quant_fp8_cols_kernel<__bf16> : (const void *)quant_fp8_rows_kernel<__bf16>;
    else fn = transpose ? (const void *)quant_fp8_cols_kernel<float> : (const void *)quant_fp8_rows_kernel<float>;
    QuantFp8Args arg = a;
    void *args[] = {&arg};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)grid, 1, 1), dim3(256, 1, 1), args, 0, s);
    return e != hipSuccess ? e : hipGetLastError();
}

}  // namespace dg
