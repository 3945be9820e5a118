// moe.hip - tokens sorted by expert, and the movement of their rows to the
// experts and back, with the router's weights and its gradient.
//
// A pair is one choice of a token, pair = token * topk + slot.  The sort puts the
// pairs of expert e into rows off[e] .. off[e+1]-1, in pair order, each expert's
// rows rounded up to `align`; src[row] is a row's pair (or -1) and dst[pair] its
// row (or -1 for a pair whose id names no expert).
#include <algorithm>

#include "kcommon.h"
#include "moe_args.h"
#include "row8.h"

namespace dg {

// ------------------------------------------------------------------------ sort
constexpr int ST = 1024, SW = ST / 64;   // threads and waves of a sorting workgroup
constexpr int SORT_BLOCKS = 256;         // most workgroups

// Sum over lanes 0 .. lane of the workgroup (inclusive); s_part: SW ints.
DG_DEV int block_scan(int v, int *s_part)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    if (lane == 63) s_part[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += s_part[w];
    __syncthreads();
    return v;
}

// Counts of each workgroup's pairs by expert: ws[block][experts].  (The LDS
// additions are of whole numbers: their order does not matter.)
__global__ void __launch_bounds__(ST) moe_count_kernel(MoeSortArgs p)
{
    __shared__ int s_n[MOE_MAX_EXPERTS];
    for (int e = threadIdx.x; e < p.experts; e += ST) s_n[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * p.per_block, hi = min((int64_t)p.pairs, lo + p.per_block);
    for (int64_t i = lo + threadIdx.x; i < hi; i += ST) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.experts) atomicAdd(&s_n[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += ST) p.ws[(int64_t)blockIdx.x * p.experts + e] = s_n[e];
}

// Latency-bound: 131072 pairs over 128 experts 2.4 us of counting and 7.8 of sorting
// (13.8 with the counts of all blocks read one by one and padding written by one
// thread an expert); 32 pairs 3.9 us.
// Every workgroup derives all offsets from the counts (its own, if it is the only
// one), then ranks its pairs 1024 at a time: inside a wave by comparing the ids'
// bits through ballots, across waves by a running count per expert.
__global__ void __launch_bounds__(ST) moe_sort_kernel(MoeSortArgs p)
{
    __shared__ int s_total[MOE_MAX_EXPERTS], s_next[MOE_MAX_EXPERTS];   // counts; the next free row of each expert
    __shared__ int s_pad[MOE_MAX_EXPERTS];
    __shared__ int s_part[SW];
    extern __shared__ int s_wave[];                                     // [SW][experts]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.experts;
    const int64_t lo = (int64_t)blockIdx.x * p.per_block, hi = min((int64_t)p.pairs, lo + p.per_block);
    int ahead = lo + tid < hi ? p.ids[lo + tid] : -1;   // the next pair's id
    for (int e = tid; e < E; e += ST) s_total[e] = s_next[e] = 0;
    __syncthreads();
    if (p.blocks == 1) {
        for (int64_t i = lo + tid; i < hi; i += ST) {
            const int e = p.ids[i];
            if (e >= 0 && e < E) atomicAdd(&s_total[e], 1);
        }
    } else {
        // counts of all blocks, and of the blocks before this one: `groups` threads
        // share an expert, each with every groups-th block, eight loads at a time
        const int groups = ST / E, g = tid / E, e = tid - g * E;
        if (g < groups) {
            int total = 0, before = 0;
            for (int b0 = g; b0 < p.blocks; b0 += 8 * groups) {
                int n[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] = p.ws[(int64_t)min(b0 + i * groups, p.blocks - 1) * E + e];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int b = b0 + i * groups;
                    total += b < p.blocks ? n[i] : 0;
                    before += b < (int)blockIdx.x ? n[i] : 0;
                }
            }
            atomicAdd(&s_total[e], total);
            atomicAdd(&s_next[e], before);
        }
    }
    __syncthreads();
    // offsets: one thread per expert
    const int n = tid < E ? s_total[tid] : 0;
    const int padded = (n + p.align - 1) / p.align * p.align;
    const int end = block_scan(padded, s_part), first = end - padded;
    if (tid < E) {
        s_next[tid] += first;
        if (blockIdx.x == 0) {
            p.off[tid + 1] = end;
            if (tid == 0) p.off[0] = 0;
        }
    }
    if (tid == ST - 1) s_part[0] = end;   // rows in all segments
    __syncthreads();
    const int used = s_part[0];
    // rows without a pair: the padding of this workgroup's experts, one wave each
    // (the ends meet in s_total and s_pad), and the tail
    if (tid < E) s_total[tid] = first + n, s_pad[tid] = end;
    __syncthreads();
    for (int x = (int)blockIdx.x + wave * p.blocks; x < E; x += SW * p.blocks)
        for (int r = s_total[x] + lane; r < s_pad[x]; r += 64) p.src[r] = -1;
    for (int64_t r = used + (int64_t)blockIdx.x * ST + tid; r < p.capacity; r += (int64_t)p.blocks * ST) p.src[r] = -1;
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    for (int64_t base = lo; base < hi; base += ST) {
        const int64_t i = base + tid;
        const int e = ahead < E ? ahead : -1;
        ahead = i + ST < hi ? p.ids[i + ST] : -1;
        for (int x = lane; x < E; x += 64) s_wave[wave * E + x] = 0;   // (this wave's own counts)
        unsigned long long same = __ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const unsigned long long one = __ballot(e >> b & 1);
            same &= (e >> b & 1) ? one : ~one;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && rank == 0) s_wave[wave * E + e] = __popcll(same);
        __syncthreads();
        for (int x = tid; x < E; x += ST) {   // each wave's first row of each expert
            int at = s_next[x], c[SW];
#pragma unroll
            for (int w = 0; w < SW; ++w) c[w] = s_wave[w * E + x];
#pragma unroll
            for (int w = 0; w < SW; ++w) {
                s_wave[w * E + x] = at;
                at += c[w];
            }
            s_next[x] = at;
        }
        __syncthreads();
        if (i < hi) {
            const int row = e >= 0 ? s_wave[wave * E + e] + rank : -1;
            p.dst[i] = row;
            if (row >= 0 && row < p.capacity) p.src[row] = (int)i;
        }
        __syncthreads();
    }
}

void moe_sort_shape(int64_t pairs, int &blocks, int &per_block)
{
    int64_t b = (pairs + ST - 1) / ST;
    if (b <= 4) b = 1;
    if (b > SORT_BLOCKS) b = SORT_BLOCKS;
    const int64_t each = (pairs + b - 1) / (b ? b : 1);
    per_block = (int)((each + ST - 1) / ST * ST);
    if (per_block == 0) per_block = ST;
    blocks = (int)((pairs + per_block - 1) / per_block);
    if (blocks < 1) blocks = 1;
}

hipError_t launch_moe_sort(const MoeSortArgs &a, hipStream_t s)
{
    MoeSortArgs arg = a;
    void *args[] = {&arg};
    hipError_t e;
    if (a.blocks > 1) {
        e = hipLaunchKernel(reinterpret_cast<const void *>(moe_count_kernel), dim3(a.blocks, 1, 1), dim3(ST, 1, 1), args, 0, s);
        if (e != hipSuccess) return e;
    }
    e = hipLaunchKernel(reinterpret_cast<const void *>(moe_sort_kernel), dim3(a.blocks, 1, 1), dim3(ST, 1, 1), args,
                        (size_t)SW * a.experts * sizeof(int), s);
    return e != hipSuccess ? e : hipGetLastError();
}

// ------------------------------------------------------------ movement of rows
// A wave moves 512 columns of one row, eight per lane.  Bound by memory: 8192 tokens of
// 4096 bf16, two experts each, combine in 29.7 us with the rows in the last cache
// and 37.3 from memory (201 MB, 5.4 TB/s).
namespace {
constexpr int MV = 512;

DG_DEV float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}
}  // namespace

// out[r] = x[src[r] / topk], zeros where src names no pair
template <typename T>
__global__ void __launch_bounds__(256) moe_gather_kernel(MoeMoveArgs p)
{
    const int chunks = (p.hidden + MV - 1) / MV;
    const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t r = u / chunks;
    const int c = (int)(u - r * chunks) * MV + (threadIdx.x & 63) * 8;
    if (r >= p.rows || c >= p.hidden) return;
    const int i = p.src[r], n = p.hidden - c;
    const int t = i < 0 ? -1 : i / p.topk;
    const bool live = t >= 0 && t < p.tokens;
    const auto v = ld8(reinterpret_cast<const T *>(p.x) + t * p.ldx + c, live ? n : 0);
    st8(reinterpret_cast<T *>(p.out) + r * p.ldout + c, n, wide8<T>(v));
}

// out[t] = sum over slots of w[t][s] * x[dst[t][s]], added in slot order; the rows
// of four slots are loaded together
template <typename T>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeMoveArgs p)
{
    const int chunks = (p.hidden + MV - 1) / MV;
    const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t t = u / chunks;
    const int c = (int)(u - t * chunks) * MV + (threadIdx.x & 63) * 8;
    if (t >= p.tokens || c >= p.hidden) return;
    const int n = p.hidden - c;
    floatx8 acc = 0.f;
    for (int s0 = 0; s0 < p.topk; s0 += 4) {
        int r[4];
        float w[4];
        typename Row8<T>::vec v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = t * p.topk + min(s0 + i, p.topk - 1);
            r[i] = p.dst[at];
            w[i] = p.w ? p.w[at] : 1.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (s0 + i >= p.topk || r[i] >= p.rows) r[i] = -1;
            v[i] = ld8(reinterpret_cast<const T *>(p.x) + (int64_t)r[i] * p.ldx + c, r[i] >= 0 ? n : 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (r[i] < 0) continue;   // (a slot without a row: its weight may be anything)
            const floatx8 x = wide8<T>(v[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(w[i], x[e], acc[e]);
        }
    }
    st8(reinterpret_cast<T *>(p.out) + t * p.ldout + c, n, acc);
}

// Gradient of the combination: out[dst[t][s]] = w[t][s] dout[t] and
// dw[t][s] = <x[dst[t][s]], dout[t]>.  Wave u takes pair u, whose row it walks in
// runs of 2048 columns (1024 of binary32) with all loads of a run in flight, and then clears row u
// (and u + waves, ...) if no pair has it.  7108 rows of 1112 f16: 7.8 us (36 MB, 4.5
// TB/s; one workgroup per pair, and 64 empty rows to a wave, took 24.7).
template <typename T>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(MoeMoveArgs p)
{
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    const int lane = threadIdx.x & 63;
    const int64_t pairs = (int64_t)p.tokens * p.topk, waves = (int64_t)gridDim.x * 4;
    const int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (u < pairs) {
        const int64_t t = u / p.topk;
        const int r = p.dst[u];
        float sum = 0.f;
        if (r >= 0 && r < p.rows) {
            const float w = p.w ? p.w[u] : 1.f;
            const T *x = reinterpret_cast<const T *>(p.x) + (int64_t)r * p.ldx;
            const T *d = reinterpret_cast<const T *>(p.dout) + t * p.ld_dout;
            T *o = reinterpret_cast<T *>(p.out) + (int64_t)r * p.ldout;
            for (int c0 = lane * 8; c0 < p.hidden; c0 += U * MV) {
                typename Row8<T>::vec g[U], v[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int c = c0 + i * MV;
                    g[i] = ld8(d + c, p.hidden - c);
                    v[i] = ld8(x + c, p.dw ? p.hidden - c : 0);
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int c = c0 + i * MV;
                    const floatx8 a = wide8<T>(g[i]), b = wide8<T>(v[i]);
                    floatx8 q;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sum = __builtin_fmaf(b[e], a[e], sum);
                        q[e] = w * a[e];
                    }
                    st8(o + c, p.hidden - c, q);
                }
            }
        }
        if (p.dw) {
            sum = wave_sum(sum);
            if (lane == 0) p.dw[u] = sum;
        }
    }
    for (int64_t r = u; r < p.rows; r += waves) {
        const int i = p.src[r];
        if (i >= 0 && i < pairs) continue;
        T *o = reinterpret_cast<T *>(p.out) + r * p.ldout;
        for (int c = lane * 8; c < p.hidden; c += MV) st8(o + c, p.hidden - c, floatx8(0.f));
    }
}

namespace {
hipError_t launch_move(const void *f16, const void *bf16, const void *f32, const MoeMoveArgs &a, int64_t grid, hipStream_t s)
{
    if (grid == 0) return hipSuccess;
    if (!grid_fits(grid, 256)) return hipErrorInvalidConfiguration;
    MoeMoveArgs arg = a;
    void *args[] = {&arg};
    const void *fn = a.type == T_F16 ? f16 : (a.type == T_BF16 ? bf16 : f32);
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)grid, 1, 1), dim3(256, 1, 1), args, 0, s);
    return e != hipSuccess ? e : hipGetLastError();
}
int64_t chunk_grid(int64_t rows, int hidden) { return (rows * ((hidden + MV - 1) / MV) + 3) / 4; }
}  // namespace

hipError_t launch_moe_gather(const MoeMoveArgs &a, hipStream_t s)
{
    return launch_move((const void *)moe_gather_kernel<_Float16>, (const void *)moe_gather_kernel<__bf16>,
                       (const void *)moe_gather_kernel<float>, a, chunk_grid(a.rows, a.hidden), s);
}
hipError_t launch_moe_combine(const MoeMoveArgs &a, hipStream_t s)
{
    return launch_move((const void *)moe_combine_kernel<_Float16>, (const void *)moe_combine_kernel<__bf16>,
                       (const void *)moe_combine_kernel<float>, a, chunk_grid(a.tokens, a.hidden), s);
}
hipError_t launch_moe_combine_grad(const MoeMoveArgs &a, hipStream_t s)
{
    return launch_move((const void *)moe_combine_grad_kernel<_Float16>, (const void *)moe_combine_grad_kernel<__bf16>,
                       (const void *)moe_combine_grad_kernel<float>, a,
                       (std::max((int64_t)a.tokens * a.topk, (int64_t)a.rows) + 3) / 4, s);
}

}  // namespace dg
