// Joining the partial results of attention over parts of the keys.
#pragma once

#include "attend.hpp"

namespace fp8q {

// A unit (rows of one key/value head of a sequence) that `parts` workgroups have parts of; 0: none.
struct Unit {
    int64_t at;                           // tells units apart
    int parts, begins, ends, token0, head, row0, rows, unused;
};

// Where the partial results lie, in floats: part k of unit i at first + i * stride for k = 0, else at
// other + i * stride + k * step.  A part's rows are DP + 4 floats apart: maximum, denominator, two
// unused, sums.
struct Parts {
    const Unit* units;
    const float *first, *other;
    int64_t stride, step;
};
constexpr int kMostParts = 512;
constexpr int kJoinThreads = 256;

namespace {

// A workgroup joins R rows of a unit.  A row's threads have four channels each and take turns at
// the parts; the parts' maxima come first, so that no load waits for another.
template <int DT, int DP, int R>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a, const Parts parts)
{
    constexpr int kEach = kJoinThreads / R;
    __shared__ float stat[R][kMostParts][2];
    __shared__ __attribute__((aligned(16))) float sums[kJoinThreads * 4];
    const Unit u = parts.units[blockIdx.x];
    const int mine = threadIdx.x / kEach, tid = threadIdx.x % kEach, row = blockIdx.y * R + mine;
    if (u.parts == 0 || (int)(blockIdx.y * R) >= u.rows) return;
    const int64_t at = blockIdx.x * parts.stride + (int64_t)row * (DP + 4);
    const auto part = [&](int k) { return k == 0 ? parts.first + at : parts.other + at + k * parts.step; };
    if (row < u.rows)
        for (int k = tid; k < u.parts; k += kEach) {
            const float* p = part(k);
            stat[mine][k][0] = p[0];
            stat[mine][k][1] = p[1];
        }
    __syncthreads();
    const int quads = a.D / 4, sets = kEach / quads, set = tid / quads, d = tid % quads * 4;
    Joined j{-__builtin_inff(), 0.0f, 0.0f};
    v4f o = {0.f, 0.f, 0.f, 0.f};
    if (row < u.rows && set < sets) {
        for (int k = 0; k < u.parts; ++k) j.m = fmaxf(j.m, stat[mine][k][0]);
        j.ref = j.m == -__builtin_inff() ? 0.0f : j.m;
        for (int k = 0; k < u.parts; ++k) j.l += stat[mine][k][1] * __builtin_amdgcn_exp2f(stat[mine][k][0] - j.ref);
#pragma unroll 4
        for (int k = set; k < u.parts; k += sets)
            o += *reinterpret_cast<const v4f*>(part(k) + 4 + d) * __builtin_amdgcn_exp2f(stat[mine][k][0] - j.ref);
        *reinterpret_cast<v4f*>(&sums[4 * threadIdx.x]) = o;
    }
    __syncthreads();
    if (row >= u.rows || set != 0) return;
    for (int k = 1; k < sets; ++k) o += *reinterpret_cast<const v4f*>(&sums[4 * (threadIdx.x + k * quads)]);
    const int gr = u.row0 + row;
    store_row<DT>(a, u.token0 + gr / a.group, u.head * a.group + gr % a.group, d, o, j);
}

// `about`: the parts that a unit has, for the choice between a workgroup a row and one for several.
template <int DT, int DP>
hipError_t launch_join(const AttendArgs& a, const Parts& parts, int units, int rows, int about, hipStream_t stream)
{
    constexpr int kSeveral = DP <= 128 ? 8 : 4;
    if (about >= 8) {
        hipLaunchKernelGGL((attend_join_kernel<DT, DP, 1>), dim3(units, rows), dim3(kJoinThreads), 0, stream, a, parts);
    } else {
        hipLaunchKernelGGL((attend_join_kernel<DT, DP, kSeveral>), dim3(units, (rows + kSeveral - 1) / kSeveral),
                           dim3(kJoinThreads), 0, stream, a, parts);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace fp8q
