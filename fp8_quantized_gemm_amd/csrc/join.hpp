// Joining the partial results of attention over parts of the keys:
//   m = max m_i,  z = max z_i,  l = sum l_i 2^(z_i - z),  y = 2^(m - z) sum y_i 2^(m_i - m) / l
// A second launch of 4 to 6 us (8 rows of 64 parts each of 8 heads 5.7 us, 52 units of 35 rows in 4 parts 4.5), bound by
// the latency of two dependent rounds of loads; the parts come in a fixed order, so results repeat.
#pragma once

#include "attend.hpp"

namespace fp8q {

// A unit: rows row0 .. of a key/value head of a sequence (its first token's row: token0), which
// `parts` workgroups have parts of, the first of them workgroup `group`; parts = 0: none.
struct Unit {
    int group, parts, token0, head, row0, rows, unused[2];
};

// The parts of a unit are those of every Hk-th workgroup from its first on.  A part's rows are DP + 4
// floats apart: the sums' reference m, the denominator l and its reference z, one unused, sums y.
constexpr int kMostParts = 512;
constexpr int kJoinThreads = 256;

namespace {

// A workgroup joins R rows of a unit.  A row's threads have four channels each and take turns at
// the parts; the parts' maxima come first, so that no load waits for another.
template <int DT, int DP, int R>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a, const float* parts,
                                                                    int part_rows)
{
    constexpr int kEach = kJoinThreads / R, kLanes = kEach < 64 ? kEach : 64, kWaves = kJoinThreads / 64;
    __shared__ float factor[R][kMostParts], red[3][kWaves];
    __shared__ __attribute__((aligned(16))) float sums[kJoinThreads * 4];
    const Unit u = reinterpret_cast<const Unit*>(a.work)[blockIdx.x];
    const int mine = threadIdx.x / kEach, tid = threadIdx.x % kEach, row = blockIdx.y * R + mine;
    if (u.parts == 0 || (int)(blockIdx.y * R) >= u.rows) return;
    const int count = row < u.rows ? u.parts : 0;
    const auto part = [&](int k) {
        return parts + (((int64_t)u.group + (int64_t)k * a.Hk) * part_rows + row) * (DP + 4);
    };
    float m = -__builtin_inff(), z = m, l = 0.0f;
    for (int k = tid; k < count; k += kEach) {
        factor[mine][k] = part(k)[0];
        m = fmaxf(m, factor[mine][k]);
        z = fmaxf(z, part(k)[2]);
    }
#pragma unroll
    for (int off = kLanes / 2; off >= 1; off >>= 1) {
        m = fmaxf(m, __shfl_xor(m, off));
        z = fmaxf(z, __shfl_xor(z, off));
    }
    if constexpr (kEach > 64) {
        if ((threadIdx.x & 63) == 0) { red[0][threadIdx.x >> 6] = m; red[2][threadIdx.x >> 6] = z; }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) { m = fmaxf(m, red[0][w]); z = fmaxf(z, red[2][w]); }
    }
    const float ref = m == -__builtin_inff() ? 0.0f : m, zref = z == -__builtin_inff() ? 0.0f : z;
    for (int k = tid; k < count; k += kEach) {
        factor[mine][k] = __builtin_amdgcn_exp2f(factor[mine][k] - ref);
        l += part(k)[1] * __builtin_amdgcn_exp2f(part(k)[2] - zref);
    }
#pragma unroll
    for (int off = kLanes / 2; off >= 1; off >>= 1) l += __shfl_xor(l, off);
    if constexpr (kEach > 64) {
        if ((threadIdx.x & 63) == 0) red[1][threadIdx.x >> 6] = l;
    }
    __syncthreads();
    const int quads = a.D / 4, sets = kEach / quads, set = tid / quads, d = tid % quads * 4;
    v4f o = {0.f, 0.f, 0.f, 0.f};
    if (set < sets) {
#pragma unroll 4
        for (int k = set; k < count; k += sets)
            o += *reinterpret_cast<const v4f*>(part(k) + 4 + d) * factor[mine][k];
        *reinterpret_cast<v4f*>(&sums[4 * threadIdx.x]) = o;
    }
    __syncthreads();
    if (count == 0 || set != 0) return;
    for (int k = 1; k < sets; ++k) o += *reinterpret_cast<const v4f*>(&sums[4 * (threadIdx.x + k * quads)]);
    if constexpr (kEach > 64) l = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    const int gr = u.row0 + row;
    store_row<DT>(a, u.token0 + gr / a.group, u.head * a.group + gr % a.group, d, o, Joined{ref, zref, l});
}

template <int DT, int DP>
hipError_t launch_join(const AttendArgs& a, const float* parts, int64_t units, int part_rows, hipStream_t stream)
{
    // a workgroup a row where there are few, several rows where they fill the chip by far
    constexpr int kSeveral = DP <= 128 ? 8 : 4;
    const unsigned groups = (unsigned)(units * a.Hk);
    if ((int64_t)groups * part_rows <= 2048) {
        hipLaunchKernelGGL((attend_join_kernel<DT, DP, 1>), dim3(groups, part_rows), dim3(kJoinThreads), 0, stream, a,
                           parts, part_rows);
    } else {
        hipLaunchKernelGGL((attend_join_kernel<DT, DP, kSeveral>), dim3(groups, (part_rows + kSeveral - 1) / kSeveral),
                           dim3(kJoinThreads), 0, stream, a, parts, part_rows);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace fp8q
