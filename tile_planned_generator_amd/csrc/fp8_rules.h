// fp8_rules.h - host-side rules of the block-scaled fp8 products.  Plain C++ without
// HIP, so that they can be checked on a machine without a GPU.
#pragma once
#include <cstdint>

namespace dg {

// Whether `experts` matrices of M x N elements, rows ld apart and matrices `stride`
// apart, share no element: whole matrices one after the other, or the matrices'
// rows interleaved inside one row pitch.  (128 bits: the caller's pitches are not bounded.)
inline bool experts_disjoint(int64_t M, int64_t N, int64_t ld, int64_t stride, int64_t experts)
{
    if (experts <= 1 || M <= 0 || N <= 0) return true;
    const __int128 span = (__int128)(M - 1) * ld + N;
    return stride >= span || (stride >= N && ld >= (__int128)(experts - 1) * stride + N);
}

// Whether every byte of `rows` rows of K bytes, ld apart, has an offset below 2^32: the
// kernels count bytes from a tile's origin in 32 bits.  (Divided, as ld * rows may
// pass 64 bits: pitches from 2^57 on would look small.)
inline bool rows_fit_32(int rows, int64_t ld, int64_t K)
{
    const int64_t last = (int64_t(1) << 32) - 1;
    return K <= last && ld <= (last - K) / rows;
}

}  // namespace dg
