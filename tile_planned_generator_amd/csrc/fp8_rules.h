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

}  // namespace dg
