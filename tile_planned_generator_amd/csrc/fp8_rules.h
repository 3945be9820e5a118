// fp8_rules.h - host-side rules of the block-scaled fp8 products: which kernel takes a
// problem, and what it can address.  Plain C++ without HIP, so that they can be
// checked on a machine without a GPU.
#pragma once
#include <algorithm>
#include <cstdint>

namespace dg {

constexpr int FP8_BLOCK = 128;   // values along K that share a scale
// The largest size of the expert layer's calls: launchers and kernels round sizes up to
// whole tiles, blocks and runs (of 2048 columns at most) in 32 bits.
constexpr int64_t FP8_MOST = INT32_MAX - 4095;
// Kernel variants of the product (indices of the tables in gemm_fp8.hip).
enum Fp8Kernel : int { FP8_STREAM16 = 0, FP8_TILE64, FP8_TILE128, FP8_TILE256, FP8_KERNELS };

// Whether one launch takes so many workgroups: HIP counts a launch's work-items in 32
// bits along x.  (128 bits: tiles times experts may pass 64.)
inline bool grid_fits(__int128 workgroups, int threads) { return workgroups * threads < (__int128)1 << 32; }

inline int64_t blocks_of(int64_t n) { return (n + FP8_BLOCK - 1) / FP8_BLOCK; }

struct Fp8Choice {
    int kernel, split;
};

inline int64_t tiles_of(int64_t M, int64_t N, int t) { return ((M + t - 1) / t) * ((N + t - 1) / t); }

// Whether every byte of `rows` rows of K bytes, ld apart, has an offset below 2^32: the
// kernels count bytes from a tile's origin in 32 bits.  (Divided, as ld * rows may
// pass 64 bits: pitches from 2^57 on would look small.)
inline bool rows_fit_32(int rows, int64_t ld, int64_t K)
{
    const int64_t last = (int64_t(1) << 32) - 1;
    return K <= last && ld <= (last - K) / rows;
}

// Whether the 256 x 256 tile can take a product: the exact products of binary32 outputs
// leave it no registers, and the 256 rows of an operand that it addresses have to lie
// within 32 bits (a row pitch below about 16 MiB; the other tiles address 128).
inline bool huge_tile(bool exact, int64_t lda, int64_t ldb, int64_t K)
{
    return !exact && rows_fit_32(256, lda, K) && rows_fit_32(256, ldb, K);
}

// The tile for `wide` 128 x 128 tiles or `huge` 256 x 256 ones.  Fewer than 256 wide
// ones leave CUs idle, and 64 x 64 ones are faster (768 rows over 8 experts,
// N = 2048, K = 4096: 19.3 against 27.0 us; 512 rows, N = 4096 dense: 17.9 against
// 23.9; 1024 rows, 256 wide tiles: 31.6 against 25.9).  A chip full of 256 x 256
// tiles (one to a CU) takes as long as 768 wide ones (two to a CU): 4096^3 is one
// round of them, 61.7 against 73.4 us, 16384 rows over 8 experts, N = 2048, would be
// three short ones, 167 against 156.
inline int tiled_kernel(int64_t wide, int64_t huge, bool huge_ok)
{
    if (wide < 256) return FP8_TILE64;
    return huge_ok && (huge + 255) / 256 * 768 <= wide ? FP8_TILE256 : FP8_TILE128;
}

// Up to 16 rows stream B through registers (N = K = 4096: 9.0 against 12.4 us for 64 x
// 64 tiles and a K split); from 17 on the tiles are as fast (32 rows, 12.8 us).
inline Fp8Choice choose_dense(int64_t M, int64_t N, int64_t K, bool huge_ok)
{
    if (M <= 16) return {FP8_STREAM16, 1};
    const int kernel = tiled_kernel(tiles_of(M, N, 128), tiles_of(M, N, 256), huge_ok);
    if (kernel != FP8_TILE64) return {kernel, 1};
    const int64_t tiles = tiles_of(M, N, 64), steps = blocks_of(K);
    // too few tiles for 256 CUs: cut K, in slices of at least four steps
    int64_t split = 1;
    if (tiles > 0 && tiles < 192) split = std::max<int64_t>(1, std::min<int64_t>(steps / 4, 512 / tiles));
    return {kernel, (int)std::min<int64_t>(split, 32)};
}

// Row tiles to expect: an expert's rows end inside a tile, on average half way.
inline int64_t row_tiles(int64_t rows, int64_t experts, int64_t bm)
{
    return rows >= experts * bm ? rows / bm + experts / 2 : std::min(rows, experts);
}

// With experts the 64 x 64 tiles win at few rows too, as their loads run three steps
// ahead (B out of every cache, 16-bit output, 8 experts of 4096 x 4096: 4 rows each
// 27.9 us, streamed 38.0, as 128 x 128 tiles 38.9; of 2048 x 4096: 16 rows 18.4
// against 30.0 streamed), but for the exact products of four rows or fewer (1 row
// 20.6 against 11.8 us, 4 rows 21.2 against 20.1, 12 rows 21.3 against 27.5).
inline int choose_rows(int64_t rows, int64_t experts, int64_t N, bool exact, bool huge_ok)
{
    if (exact && rows <= 4 * experts) return FP8_STREAM16;
    if (rows <= 64 * experts) return FP8_TILE64;
    return tiled_kernel(row_tiles(rows, experts, 128) * ((N + 127) / 128),
                        row_tiles(rows, experts, 256) * ((N + 255) / 256), huge_ok);
}

inline int choose_wgrad(int64_t M, int64_t N, int64_t experts, bool huge_ok)
{
    return tiled_kernel(tiles_of(M, N, 128) * experts, tiles_of(M, N, 256) * experts, huge_ok);
}

// K slices of whole blocks; the count after rounding the slices up.
inline void slices(int64_t K, int split, int &k_slice, int &count)
{
    const int64_t steps = std::max<int64_t>(1, blocks_of(K)), each = (steps + split - 1) / split;
    k_slice = (int)(each * FP8_BLOCK);
    count = (int)((steps + each - 1) / each);
}

// Whether `experts` matrices of M x N elements, rows ld apart and matrices `stride`
// apart, share no element: whole matrices one after the other, or the matrices'
// rows interleaved inside one row pitch.  (128 bits: the caller's pitches are not bounded.)
inline bool experts_disjoint(int64_t M, int64_t N, int64_t ld, int64_t stride, int64_t experts)
{
    if (experts <= 1 || M <= 0 || N <= 0) return true;
    const __int128 span = (__int128)(M - 1) * ld + N;
    return stride >= span || (stride >= N && ld >= (__int128)(experts - 1) * stride + N);
}

}  // namespace dg
